"""Norms of finite rows anywhere in fp32's range, against the fp64 oracle: rows whose squares or whose sum of squares
fp32 cannot hold, beside ordinary ones in the same call.

Tolerances are those of test_gpu_layer.py's docstring (the statistics of such rows are held in more bits, not fewer), and where
numbers are subnormal, half a step there: 2^-150 for fp32, 2^-134 for bf16.  A norm's product v w may be one while the output is
not: its half step is then multiplied by the root, which is at most 2^50 where the product is formed in fp32.
"""
import numpy as np
import pytest
import torch

import block_sparse_cluster_b200 as da
import oracle
from tests.test_gpu_layer import BF16, F32, _close, _cuda, _gen, _half, _rope_check

pytestmark = pytest.mark.gpu

# powers of two of the rows: squares below fp32's smallest number, subnormal ones, the sums' borders, sums above the largest
EXPONENTS = [0, -146, -130, -110, -75, -66, -60, -52, -50, -49, -48, 3, 55, 57, 59, 62, 63, 64, 70, 100, 122, 0]


def _rows(width, dtype, seed):
    g = _gen(seed)
    power = torch.tensor([2.0 ** e for e in EXPONENTS], dtype=torch.float64)[:, None]
    x = torch.randn(len(EXPONENTS), width, generator=g, dtype=torch.float64).clamp(-8, 8) * power
    r = torch.randn(len(EXPONENTS), width, generator=g, dtype=torch.float64).clamp(-8, 8) * power
    w = 1 + 0.2 * torch.randn(width, generator=g, dtype=torch.float64)
    return x.to(dtype), r.to(dtype), w.to(dtype)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e20, 3e38])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [1, 64, 77, 512, 1536, 2056, 4100, 5120, 9002, 16383, 16384])
def test_norm_of_rows_of_any_size(width, dtype, eps):
    x, r, w = _rows(width, dtype, width)
    rows = x.shape[0]
    for residual, weight in ((None, None), (r, w)):
        xc, rc, wc = x.cuda(), _cuda(residual), _cuda(weight)
        out, total = torch.empty_like(xc), None if residual is None else torch.empty_like(xc)
        da.da_rms_norm(xc, wc, out, residual=rc, sum_out=total, eps=eps)
        with np.errstate(divide="ignore", invalid="ignore"):
            ref, v = oracle.rms_norm(x, residual, weight, eps)
            root = np.minimum(1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps), 2.0 ** 50)
        some = np.isfinite(ref).all(-1) & (np.abs(v).max(-1) > 0)       # eps = 0 and a row of nothing but zeros: 0 / 0
        assert some.sum() >= rows - 2
        tol = np.abs(ref) * (2.0 ** -19 + _half(dtype) * 1.001) + _half_step_of_least(dtype) + 2.0 ** -150 * root
        _close(out[torch.from_numpy(some)], ref[some], tol[some])
        q, scale = torch.empty(rows, width, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        total2 = None if residual is None else rc                       # the residual stream in place
        da.da_rms_norm_i8(xc, wc, q, scale, residual=rc, sum_out=total2, eps=eps)
        with np.errstate(divide="ignore", invalid="ignore"):
            rq, rs, _ = oracle.rms_norm_i8(x, residual, weight, eps)
        rs = np.where(np.abs(v).max(-1) > 0, rs, 0.0)                   # a row of zeros has scale 0
        assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
        _close(scale, rs, rs * 2.0 ** -19 + 2.0 ** -149)
        if residual is not None:
            assert torch.equal(total2, total)
            _close(total, v, np.abs(v) * _half(dtype) * 1.001 + 2.0 ** -24 * np.abs(v) + _half_step_of_least(dtype))


def _half_step_of_least(dtype):
    """Half a step of the type's subnormal numbers, and of fp32's for the value that is rounded to it."""
    return 2.0 ** -134 + 2.0 ** -150 if dtype == BF16 else 2.0 ** -149


@pytest.mark.parametrize("width", [64, 16384])
def test_sums_beyond_fp32_at_any_width(width):
    """One element that overflows by its own square, and many that do so together."""
    x = torch.full((3, width), 1.5e17)
    x[1] = 0
    x[1, 5] = 3e20
    x[2] = 1.0
    q, scale, out = torch.empty(3, width, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, width, device="cuda")
    da.da_rms_norm_i8(x.cuda(), None, q, scale)
    da.da_rms_norm(x.cuda(), None, out)
    rq, rs, _ = oracle.rms_norm_i8(x)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    _close(scale, rs, rs * 2.0 ** -19)
    ref = oracle.rms_norm(x)[0]
    _close(out, ref, np.abs(ref) * 2.0 ** -18)


@pytest.mark.parametrize("width", [64, 77, 4096])
def test_products_below_fp32(width):
    """A weight so small that v * w is no fp32 number, though the output is."""
    g = _gen(width)
    x = torch.randn(4, width, generator=g) * torch.tensor([1e-30, 1e-25, 1e-20, 1e-38])[:, None]
    w = (1 + torch.rand(width, generator=g)) * 1e-25
    q, scale = torch.empty(4, width, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    da.da_rms_norm_i8(x.cuda(), w.cuda(), q, scale, eps=0.0)
    rq, rs, _ = oracle.rms_norm_i8(x, None, w, 0.0)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    _close(scale, rs, rs * 2.0 ** -19)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e20])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("norm", ["head", "full"])
@pytest.mark.parametrize("B,H,N,d,axes", [(1, 1, 44, 64, (32, 16, 16)), (2, 3, 23, 64, (22, 20, 22)), (1, 12, 22, 128, (44, 42, 42)), (1, 40, 22, 128, (16, 56, 56)),
                                          (1, 128, 22, 128, (42, 44, 42))])
def test_rope_after_a_norm_of_any_size(B, H, N, d, axes, norm, dtype, eps):
    """Heads (or whole tokens, where the norm is over all heads) of every size side by side."""
    g = _gen(H)
    power = torch.tensor([2.0 ** e for e in EXPONENTS], dtype=torch.float64)
    n, h = torch.arange(N)[:, None], torch.arange(H)[None]
    which = (n + (0 if norm == "full" else 5) * h) % len(EXPONENTS)
    x = torch.randn(B, H, N, d, generator=g, dtype=torch.float64).clamp(-8, 8) * power[which.expand(N, H)].T[None, :, :, None]
    x = x.to(dtype).cuda()
    weight = (1 + 0.2 * torch.randn(d if norm == "head" else H * d, generator=g)).to(dtype).cuda()
    for pairing in ("adjacent", "halves"):
        rope = da.Rope(axes=axes, grid=(2, 2, 5), pairing=pairing)      # the tokens behind the grid are normed only
        out = torch.empty_like(x)
        da.da_rope(x, out, rope, weight=weight, eps=eps)
        zero = (x == 0).all(-1) if norm == "head" else (x == 0).all(-1).all(1, keepdim=True).expand(B, H, N)
        if eps == 0:                                                    # 0 / 0
            assert torch.isnan(out[zero]).all()
            out[zero] = 0
        with np.errstate(divide="ignore", invalid="ignore"):
            _rope_check(x, out, rope, None, weight, max(eps, 1e-300), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [64, 77, 1002, 1536, 4100, 9002, 16384])
def test_wide_rows_in_place(width, dtype):
    """The norm's output and its sum in the inputs' buffers, either way round, and the codes' sum in x: the bits of separate buffers."""
    x, r, w = (t.cuda() for t in _rows(width, dtype, width + 1))
    out, total = torch.empty_like(x), torch.empty_like(x)
    da.da_rms_norm(x, w, out, residual=r, sum_out=total, eps=0.0)
    for out_is_x in (True, False):
        xc, rc = x.clone(), r.clone()
        da.da_rms_norm(xc, w, xc if out_is_x else rc, residual=rc, sum_out=rc if out_is_x else xc, eps=0.0)
        got_out, got_sum = (xc, rc) if out_is_x else (rc, xc)
        assert torch.equal(got_out.nan_to_num(7.0), out.nan_to_num(7.0)) and torch.equal(got_sum, total)
    q, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(x.shape[0], device="cuda")
    q2, scale2 = torch.empty_like(q), torch.empty_like(scale)
    da.da_rms_norm_i8(x, w, q, scale, residual=r, sum_out=total, eps=0.0)
    xc = x.clone()
    da.da_rms_norm_i8(xc, w, q2, scale2, residual=r, sum_out=xc, eps=0.0)
    assert torch.equal(q, q2) and torch.equal(scale, scale2) and torch.equal(xc, total)


@pytest.mark.parametrize("B,H,N,d,norm,dtype", [
    (1, 12, 19003, 128, "full", BF16), (1, 40, 19003, 128, "full", BF16), (2, 12, 9507, 128, "head", BF16), (1, 8, 76001, 128, "head", BF16),
    (1, 4, 76003, 128, "full", BF16), (1, 12, 19001, 128, "full", F32), (1, 3, 38001, 64, "head", F32), (1, 70, 9601, 128, "full", F32),
])
def test_rope_of_long_runs_with_values_of_any_size(B, H, N, d, norm, dtype):
    """A third of the heads or tokens outside fp32's squares, anywhere in a run: short calls' bits, the oracle's values, and in place."""
    g = _gen(N)
    rope = da.Rope(axes=(44, 42, 42) if d == 128 else (20, 22, 22), pairing="halves" if H == 12 else "adjacent")
    power = torch.tensor([1.0, 2.0 ** 80, 2.0, 2.0 ** -90, 0.5, 3.0])
    which = torch.randint(0, 6, (B, 1 if norm == "full" else H, N, 1), generator=g)
    buf = torch.randn(B, N, 2, H, d, generator=g).to(dtype).cuda()
    x = buf[:, :, 0].permute(0, 2, 1, 3)
    x.mul_(power.cuda()[which.cuda()].to(dtype))
    weight = (1 + 0.2 * torch.randn(d if norm == "head" else H * d, generator=g)).to(dtype).cuda()
    pos = torch.randint(-5000, 1 << 20, (N, 3), generator=g, dtype=torch.int32).cuda()
    out = torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    da.da_rope(x, out, rope, positions=pos, weight=weight, eps=0.0)
    some = torch.cat([torch.arange(40), torch.randint(0, N, (40,), generator=g), N - 1 - torch.arange(40)]).unique().cuda()
    _rope_check(x[:, :, some], out[:, :, some], rope, pos[some].contiguous(), weight, 0.0, dtype)
    for lo in range(0, N, 1000):
        hi = min(lo + 1000, N)
        part = torch.empty(B, H, hi - lo, d, dtype=dtype, device="cuda")
        da.da_rope(x[:, :, lo:hi], part, rope, positions=pos[lo:hi].contiguous(), weight=weight, eps=0.0)
        assert torch.equal(part, out[:, :, lo:hi]), lo
    other = buf[:, :, 1].clone()
    da.da_rope(x, x, rope, positions=pos, weight=weight, eps=0.0)
    assert torch.equal(x, out) and torch.equal(buf[:, :, 1], other)
