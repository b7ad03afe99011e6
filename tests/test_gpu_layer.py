"""The layer operators on the GPU against the fp64 oracle.

Tolerances, with u = 2^-24 (half a step of fp32) and h(t) = finfo(t).eps / 2 (half a step of the output type):

* norm: v = x + r is off by u; the sum of squares, all terms positive, by u for each level of its tree
  (at most 16 in a thread, 5 in a warp, 5 over warps) and 3u a term; mean, eps and the root's argument 2u more,
  halved by the root; rsqrtf is within 2 ulp = 4u; two products 2u, v itself u.  Together (16 + 5 + 5 + 3 + 2) / 2 + 4 + 2 + 1
  < 23u; 2^-19 = 32u is allowed, relative to each element, plus the output's rounding h.
* scale: the same root, the maximum of fp32 products (2u), times 1/127 (2u): 2^-19.
* codes: equal, every one.
* product: the integer sum is exact, its conversion, the token's scale and the fused multiply-add round once each:
  3u of |p| (p the scaled sum without bias) and the output's rounding h.
* rotation: the angle in half turns is at most 1 and rounds to fp32 with 2^-25, pi 2^-25 = 1.6u in the angle; sin and cos
  are within 1 ulp (2u at most); products and sum round once each.  7u (|a| + |b|), after a norm 23u more: 2^-18 = 64u of
  |a| + |b| is allowed, plus h.  Positions stay below 2^24, where the oracle's fp64 angles lose less than 2^-25.
"""
import numpy as np
import pytest
import torch

import block_sparse_cluster_b200 as da
import oracle

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _f64(t):
    return oracle._f64(t)


def _close(got, ref, tol):
    got, ref = _f64(got), np.asarray(ref)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) - tol):.3g} beyond, at {np.argwhere(bad)[0]}"


def _norm_close(got, ref, dtype):
    _close(got, ref, np.abs(ref) * (2.0 ** -19 + _half(dtype) * 1.001) + 1e-37)


# ---------------------------------------------------------------------------
# norm and its codes

WIDTHS = [1, 2, 7, 8, 64, 97, 128, 130, 255, 257, 258, 512, 1000, 1001, 1002, 1024, 1536, 2056, 2132, 4098, 4100, 5120, 8192, 8198, 16380, 16382, 16383, 16384]


def _rows_case(rows, width, dtype, residual, seed):
    g = _gen(seed)
    x = torch.randn(rows, width, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    x[:, ::37] *= 9.0
    r = torch.randn(rows, width, generator=g) * 2 if residual else None
    w = 1 + 0.2 * torch.randn(width, generator=g)
    return x.to(dtype), None if r is None else r.to(dtype), w.to(dtype)


def _cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_and_codes(width, dtype):
    for rows, residual, weight in ((1, False, True), (5, True, True), (130 if width < 2000 else 9, True, False)):
        x, r, w = _rows_case(rows, width, dtype, residual, seed=width + rows)
        w = w if weight else None
        xc, rc, wc = _cuda(x), _cuda(r), _cuda(w)
        out = torch.empty_like(xc)
        total = torch.empty_like(xc) if residual else None
        da.da_rms_norm(xc, wc, out, residual=rc, sum_out=total, eps=1e-5)
        ref, v = oracle.rms_norm(x, r, w, 1e-5)
        _norm_close(out, ref, dtype)
        if residual:
            _close(total, v, np.abs(v) * _half(dtype) * 1.001 + 2.0 ** -24 * np.abs(v))
        # codes, into rows padded to 16 bytes and into packed ones
        for pitch in (-(-width // 16) * 16, width):
            q = torch.full((rows, pitch), 77, dtype=torch.int8, device="cuda")
            scale = torch.empty(rows, device="cuda")
            total2 = torch.empty_like(xc) if residual else None
            da.da_rms_norm_i8(xc, wc, q[:, :width], scale, residual=rc, sum_out=total2, eps=1e-5)
            rq, rs, _ = oracle.rms_norm_i8(x, r, w, 1e-5)
            assert np.array_equal(q[:, :width].cpu().numpy().astype(np.int64), rq)
            assert (q[:, width:] == 77).all()                   # bytes behind a row are left as they were
            _close(scale, rs, rs * 2.0 ** -19 + 1e-37)
            if residual:
                assert torch.equal(total2, total)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_strides_unaligned_rows_and_broadcast(dtype):
    width, rows = 200, 11
    g = _gen(3)
    buf = torch.randn(rows, 3 * width + 5, generator=g).to(dtype).cuda()
    for lo in (0, 1, 8, width):                                  # aligned and unaligned bases, an odd pitch
        x = buf[:, lo:lo + width]
        one = torch.randn(1, width, generator=g).to(dtype).cuda()
        r = one.expand(rows, width)                              # one residual row for all
        out = torch.full((rows, width + 24), 5.0, dtype=dtype, device="cuda")
        total = torch.full((rows, width + 3), 6.0, dtype=dtype, device="cuda")
        da.da_rms_norm(x, None, out[:, 16:16 + width], residual=r, sum_out=total[:, :width])
        ref, v = oracle.rms_norm(x.cpu(), r.cpu(), None, 1e-6)
        _norm_close(out[:, 16:16 + width], ref, dtype)
        assert (out[:, :16] == 5).all() and (out[:, 16 + width:] == 5).all() and (total[:, width:] == 6).all()


@pytest.mark.parametrize("width", [96, 1536, 1001])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_in_place(width, dtype):
    x, r, w = _rows_case(33, width, dtype, True, seed=5)
    want_out, want_sum = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    da.da_rms_norm(x.cuda(), w.cuda(), want_out, residual=r.cuda(), sum_out=want_sum)
    for out_is_x in (True, False):
        xc, rc = x.cuda(), r.cuda()
        da.da_rms_norm(xc, w.cuda(), xc if out_is_x else rc, residual=rc, sum_out=rc if out_is_x else xc)
        assert torch.equal(xc if out_is_x else rc, want_out) and torch.equal(rc if out_is_x else xc, want_sum)
    rq, rs, _ = oracle.rms_norm_i8(x, r, w)
    for into in ("x", "r"):
        xc, rc = x.cuda(), r.cuda()
        q, scale = torch.empty(33, width, dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
        da.da_rms_norm_i8(xc, w.cuda(), q, scale, residual=rc, sum_out=xc if into == "x" else rc)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
        assert torch.equal(xc if into == "x" else rc, want_sum)


@pytest.mark.parametrize("width", [64, 512, 4096, 333])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_zeros_infinities_and_nan(width, dtype):
    g = _gen(9)
    x = torch.randn(6, width, generator=g).to(dtype)
    x[1] = 0
    x[2, width // 2] = float("inf")
    x[3, width - 1] = float("nan")
    x[4, 3] = float("-inf")
    xc = x.cuda()
    q, scale, out = torch.empty(6, width, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(xc)
    for norm in (True, False):
        if norm:
            da.da_rms_norm_i8(xc, None, q, scale, eps=0.0)
            rq, rs, _ = oracle.rms_norm_i8(x[[0, 5]], None, None, 0.0)
        else:
            da.da_quantize_i8(xc, q, scale)
            rq, m = oracle.row_codes(x[[0, 5]])
            rs = m / 127
        assert np.array_equal(q[[0, 5]].cpu().numpy(), rq)
        _close(scale[[0, 5]], rs, rs * 2.0 ** -19)
        assert (q[1:5] == 0).all() and scale[1] == 0 and torch.isnan(scale[2:5]).all()
    da.da_rms_norm(xc, None, out, eps=1e-6)
    assert (out[1] == 0).all() and torch.isnan(out[3]).all()
    assert torch.isnan(out[2, width // 2]) and (out[2, : width // 2] == 0).all()     # x / inf
    _norm_close(out[[0, 5]], oracle.rms_norm(x[[0, 5]], None, None)[0], dtype)


@pytest.mark.parametrize("width", [64, 2048, 77])
def test_codes_next_to_borders(width):
    """Rows whose quotients are ties or one fp32 step beside them; rows of tiny and of huge values."""
    g = _gen(11)
    rows = []
    for base in (254.0, 127.0, 2.0 ** -120 * 254, 2.0 ** 100 * 254, 2.0 ** -140 * 254):
        k = torch.randint(-127, 128, (width,), generator=g).double()
        t = (k + 0.5).clamp(-126.5, 126.5) * (base / 127)
        t[0] = base
        rows.append(t)
        near = t.float()
        near[1:] = torch.nextafter(near[1:], torch.full((), 0.0))
        rows.append(near.double())
        near = t.float()
        near[1:] = torch.nextafter(near[1:], torch.sign(near[1:]) * 3e38)
        rows.append(near.double())
    x = torch.stack(rows).float()
    q, scale = torch.empty(len(rows), width, dtype=torch.int8, device="cuda"), torch.empty(len(rows), device="cuda")
    da.da_quantize_i8(x.cuda(), q, scale)
    rq, m = oracle.row_codes(x)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)
    _close(scale, m / 127, m / 127 * 2.0 ** -19 + 2.0 ** -149)
    # through a sum and a weight: t is formed in fp64 where fp32 cannot tell
    w = (1 + torch.rand(width, generator=g)).float()
    r = torch.randn(len(rows), width, generator=g) * x.abs().amax(1, keepdim=True) * 1e-4
    da.da_rms_norm_i8((x / w).cuda(), w.cuda(), q, scale, residual=r.cuda(), eps=0.0)
    rq, rs, _ = oracle.rms_norm_i8(x / w, r, w, 0.0)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), rq)


def test_codes_of_every_bf16_quotient():
    """Every 8-bit t against every 8-bit maximum, twelve binades down, both signs: all ties of the bf16 quantiser."""
    T = torch.arange(128, 256).double()
    t = torch.cat([T * 2.0 ** -s for s in range(12)])
    rows = []
    for M in range(128, 256):
        r = t.clone()
        r[r > M] = 0
        rows.append(torch.cat([r, -r, torch.tensor([float(M)] * 8).double()]))
    x = torch.stack(rows).to(BF16)
    for width in (x.shape[1], x.shape[1] - 3):              # by vectors and one by one
        part = x[:, -width:].contiguous()
        q, scale = torch.empty(128, width, dtype=torch.int8, device="cuda"), torch.empty(128, device="cuda")
        da.da_quantize_i8(part.cuda(), q, scale)
        ref, m = oracle.row_codes(part)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), ref)
        # the same rows as a norm's input, whose second looks settle them
        da.da_rms_norm_i8(part.cuda(), None, q, scale)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), ref)


@pytest.mark.parametrize("width", [1536, 3000, 777])
def test_codes_of_many_rows(width):
    """Thousands of rows, so that maxima that meet, ties at half the maximum and second looks all turn up."""
    g = _gen(width)
    x = torch.randn(3000, width, generator=g).to(BF16)
    r = torch.randn(3000, width, generator=g).to(BF16)
    w = (1 + 0.1 * torch.randn(width, generator=g)).to(BF16)
    q, scale = torch.empty(3000, width, dtype=torch.int8, device="cuda"), torch.empty(3000, device="cuda")
    for residual, weight in ((None, None), (r, w), (x, None)):   # the last: the residual is x itself
        xc = x.cuda()
        rc = xc if residual is x else _cuda(residual)
        da.da_rms_norm_i8(xc, _cuda(weight), q, scale, residual=rc)
        ref, _, _ = oracle.rms_norm_i8(x, residual, weight)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), ref)


def test_rows_and_heads_at_a_distance():
    """Strides whose offsets pass 32 bits, in elements and in bytes."""
    big = torch.empty(3 * (1 << 31) + 4096, dtype=BF16, device="cuda")
    step = (1 << 31) + 64
    g = _gen(4)
    x = big.as_strided((3, 512), (step, 1))
    x.copy_(torch.randn(3, 512, generator=g).to(BF16))
    q, scale, out = torch.empty(3, 512, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, 512, dtype=BF16, device="cuda")
    da.da_rms_norm(x, None, out)
    _norm_close(out, oracle.rms_norm(x.cpu())[0], BF16)
    da.da_rms_norm(out, None, x)                                 # and into far rows
    _norm_close(x, oracle.rms_norm(out.cpu())[0], BF16)
    for strides in ((0, step, 128, 1), (0, 128, step, 1)):           # heads far apart, tokens far apart
        h = big.as_strided((1, 3, 3, 128), strides)
        h.copy_(torch.randn(1, 3, 3, 128, generator=g).to(BF16))
        codes = torch.empty(3, 384, dtype=torch.int8, device="cuda")
        da.da_quantize_i8(h, codes, scale)
        ref, m = oracle.row_codes(h.cpu().permute(0, 2, 1, 3).reshape(3, 384))
        assert np.array_equal(codes.cpu().numpy().astype(np.int64), ref)
        rope, near = da.Rope((44, 42, 42), (1, 1, 3)), torch.empty(1, 3, 3, 128, dtype=BF16, device="cuda")
        da.da_rope(h, near, rope)
        _rope_check(h, near, rope, None, None, 0, BF16)
        da.da_rope(near, h, rope)
        _rope_check(near, h.contiguous(), rope, None, None, 0, BF16)


def test_strides_of_single_entries_do_not_matter():
    """torch leaves any stride on a dimension of one entry."""
    g = _gen(6)
    x = torch.randn(1, 4, 40, 64, generator=g).to(BF16).cuda()
    odd = x.as_strided(x.shape, (3, *x.stride()[1:]))
    rope = da.Rope((20, 22, 22), (1, 5, 8))
    a, b = torch.empty_like(x), torch.empty_like(x)
    da.da_rope(x, a, rope)
    da.da_rope(odd, b.as_strided(b.shape, (7, *b.stride()[1:])), rope)
    assert torch.equal(a, b)
    w, sw, s, ws = _codes(256, 64, 64, 1), _scales(256, 2).cuda(), _scales(40, 3).cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    xq = _codes(40, 64, 64, 5)
    da.da_linear_i8(xq, s, w, sw, a, ws)
    da.da_linear_i8(xq, s, w, sw, b.as_strided(b.shape, (7, *b.stride()[1:])), ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,N,d", [(1, 1, 1, 64), (2, 3, 37, 64), (1, 12, 130, 128), (3, 40, 5, 128), (2, 5, 19, 24), (1, 7, 3, 9), (2, 3, 31, 10), (1, 40, 6, 50), (1, 100, 3, 90)])
def test_quantize_heads(B, H, N, d, dtype):
    x = (torch.randn(B, H, N, d, generator=_gen(B + N)) * 3).to(dtype)
    ref, m = oracle.row_codes(x.permute(0, 2, 1, 3).reshape(B * N, H * d))
    token_major = x.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    for xc in (x.cuda(), token_major):
        q = torch.full((B * N, H * d + 16), 33, dtype=torch.int8, device="cuda")
        scale = torch.empty(B * N, device="cuda")
        da.da_quantize_i8(xc, q[:, :H * d], scale)
        assert np.array_equal(q[:, :H * d].cpu().numpy().astype(np.int64), ref) and (q[:, H * d:] == 33).all()
        _close(scale, m / 127, m / 127 * 2.0 ** -19)


# ---------------------------------------------------------------------------
# product

def _codes(rows, K, pitch, seed):
    x = torch.full((rows, pitch), 99, dtype=torch.int8)
    x[:, :K] = torch.randint(-128, 128, (rows, K), generator=_gen(seed), dtype=torch.int8)
    return x.cuda()[:, :K]


def _scales(n, seed):
    return torch.exp(0.5 * torch.randn(n, generator=_gen(seed))) * 0.01


def _linear_close(got, x, sx, w, sw, bias, dtype):
    ref, p = oracle.linear_i8(x.cpu(), sx, w.cpu(), sw, bias)
    u = 2.0 ** -24
    _close(got, ref, 3 * u * np.abs(p) + _half(dtype) * (np.abs(ref) + 3 * u * np.abs(p)) * 1.001 + 1e-37)


LINEAR = [(1, 1, 1), (1, 64, 16), (3, 17, 100), (16, 32, 128), (33, 257, 129), (64, 64, 1000), (127, 128, 256), (128, 129, 384),
          (129, 255, 144), (200, 512, 640), (257, 640, 2048), (300, 96, 5120), (513, 1537, 1000), (1, 5120, 1536), (2, 2500, 1555), (5, 601, 4111), (7, 2401, 2048), (8, 2, 15), (1000, 40, 64), (9, 48, 131),
          (2, 30720, 256), (777, 3100, 72), (2049, 384, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K", LINEAR)
def test_linear(M, C, K, dtype):
    for packed in (False, True):
        pitch = K if packed else -(-K // 16) * 16
        if packed and K % 16 == 0:
            continue                                             # the same call again
        x, w = _codes(M, K, pitch, M), _codes(C, K, pitch, C + 1)
        sx, sw = _scales(M, 3), _scales(C, 4)
        bias = torch.randn(C, generator=_gen(5)) if M % 2 else None
        out = torch.full((M, C + 8), 7.0, dtype=dtype, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:, :C], ws, bias=_cuda(bias))
        assert da.da_device_status(ws) == 0
        _linear_close(out[:, :C], x, sx, w, sw, bias, dtype)
        assert (out[:, C:] == 7).all()                           # columns behind the last one are left as they were


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,N,d,K", [(1, 1, 1, 64, 64), (2, 3, 70, 64, 256), (3, 2, 129, 128, 128), (1, 12, 300, 128, 512), (2, 5, 64, 24, 96),
                                       (5, 3, 31, 9, 80)])
def test_linear_into_heads(B, H, N, d, K, dtype):
    x, w = _codes(B * N, K, K, 1), _codes(H * d, K, K, 2)
    sx, sw, bias = _scales(B * N, 3), _scales(H * d, 4), torch.randn(H * d, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    heads = torch.full((B, H + 1, N + 2, d), 7.0, dtype=dtype, device="cuda")     # heads and tokens beyond stay as they were
    tokens = torch.full((B, N, H, d), 7.0, dtype=dtype, device="cuda")
    for out in (heads[:, :H, :N], tokens.permute(0, 2, 1, 3)):
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out, ws, bias=bias.cuda())
        flat = out.permute(0, 2, 1, 3).reshape(B * N, H * d)
        _linear_close(flat, x, sx, w, sw, bias, dtype)
    assert (heads[:, H:] == 7).all() and (heads[:, :, N:] == 7).all() and da.da_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K", [(2500, 2000, 272), (18900, 250, 1600), (4864, 1024, 128), (1100, 4096, 640)])
def test_linear_over_many_tiles(M, C, K, dtype):
    """Products of more tiles than the GPU has processors, ragged on every side; heads on the last."""
    x, w = _codes(M, K, K, 1), _codes(C, K, K, 2)
    sx, sw, bias = _scales(M, 3), _scales(C, 4), torch.randn(C, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 1, C + 8), 7.0, dtype=dtype, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:M, :C], ws, bias=bias.cuda())
    assert da.da_device_status(ws) == 0
    _linear_close(out[:M, :C], x, sx, w, sw, bias, dtype)
    assert (out[M:] == 7).all() and (out[:, C:] == 7).all()
    if C % 128 == 0:
        heads = torch.full((2, C // 128, M // 2, 128), 7.0, dtype=dtype, device="cuda")
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), heads, ws, bias=bias.cuda())
        assert torch.equal(heads.permute(0, 2, 1, 3).reshape(M, C), out[:M, :C])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K,dx,dw", [(1, 40, 3, 1, 2), (130, 200, 125, 3, 0), (129, 129, 129, 1, 1), (300, 1000, 260, 2, 3), (70, 2100, 393, 0, 1),
                                         (2600, 1300, 1001, 3, 2), (4, 5000, 1536, 1, 0), (33, 32, 128, 2, 2)])
def test_linear_rows_off_16_bytes(M, C, K, dx, dw, dtype):
    """Rows that start anywhere: odd strides, odd bases, codes of neighbouring bytes that are not the rows'; heads on the last."""
    def place(rows, offset, seed):
        flat = torch.randint(-128, 128, (rows * (K + 5) + 8,), generator=_gen(seed), dtype=torch.int8).cuda()
        return flat[offset:].as_strided((rows, K), (K + 5, 1))
    x, w = place(M, dx, 1), place(C, dw, 2)
    sx, sw, bias = _scales(M, 3), _scales(C, 4), torch.randn(C, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 1, C + 3), 7.0, dtype=dtype, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:M, :C], ws, bias=bias.cuda())
    assert da.da_device_status(ws) == 0
    _linear_close(out[:M, :C], x.contiguous(), sx, w.contiguous(), sw, bias, dtype)
    assert (out[M:] == 7).all() and (out[:, C:] == 7).all()
    aligned = torch.empty_like(out)
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % 16))[:, :K]           # the same codes in rows of 16 bytes
    da.da_linear_i8(pad(x), sx.cuda(), pad(w), sw.cuda(), aligned[:M, :C], ws, bias=bias.cuda())
    assert torch.equal(aligned[:M, :C], out[:M, :C])                 # sums are exact and the epilogues' operations the same
    if M % 2 == 0 and C % 4 == 0:
        heads = torch.full((2, 5, M // 2, C // 4), 7.0, dtype=dtype, device="cuda")
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), heads[:, :4], ws, bias=bias.cuda())
        assert torch.equal(heads[:, :4].permute(0, 2, 1, 3).reshape(M, C), out[:M, :C]) and (heads[:, 4] == 7).all()
    same = x[:1].expand(M, K)                                        # one row for every token
    da.da_linear_i8(same, sx.cuda(), w, sw.cuda(), out[:M, :C], ws)
    _linear_close(out[:M, :C], same.contiguous(), sx, w.contiguous(), sw, None, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,N,d,K", [(1, 1, 700, 601, 160), (1, 1, 45, 9, 64), (3, 2, 96, 160, 128), (2, 4, 333, 64, 256), (1, 7, 2600, 96, 128), (40, 3, 32, 48, 64),
                                       (1, 1, 6000, 1337, 128), (2, 3, 64, 80, 128)])
def test_linear_rows_stored_in_boxes(B, H, N, d, K, dtype):
    """Outputs whose rows start on 16 bytes, of any width: what lies between and behind the rows stays as it was."""
    x, w = _codes(B * N, K, K, 1), _codes(H * d, K, K, 2)
    sx, sw, bias = _scales(B * N, 3), _scales(H * d, 4), torch.randn(H * d, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pitch = -(-d // 8) * 8
    heads = torch.full((B, H + 1, N + 2, pitch), 7.0, dtype=dtype, device="cuda")
    tokens = torch.full((B, N + 1, H + 1, pitch), 7.0, dtype=dtype, device="cuda")
    flat = None
    for base, out in ((heads, heads[:, :H, :N, :d]), (tokens, tokens[:, :N, :H, :d].permute(0, 2, 1, 3))):
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out, ws, bias=bias.cuda())
        got = out.permute(0, 2, 1, 3).reshape(B * N, H * d)
        if flat is None:
            _linear_close(got, x, sx, w, sw, bias, dtype)
            flat = got.clone()
        assert torch.equal(got, flat)
        out.fill_(7)
        assert (base == 7).all() and da.da_device_status(ws) == 0


def test_linear_extremes():
    """The largest sums (every code -128 at the deepest product), codes of a row that was not finite, zero scales."""
    K = 131071
    x = torch.full((2, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((32, K + 1), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1] = 127
    sx, sw = torch.tensor([1.0, float("nan")]), torch.ones(32)
    sw[2] = 0
    out = torch.empty(2, 32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out, ws)
    assert torch.isnan(out[1]).all()
    row = out[0].cpu().double()
    assert row[0] == float(np.float32(128 * 128 * K)) and row[1] == float(np.float32(-128 * 127 * K)) and row[2] == 0


def test_linear_rows_at_a_distance():
    """Row strides whose offsets pass 32 bits, of codes and of the output."""
    M, C, K = 3, 48, 64
    step = (1 << 31) + 16
    xb = torch.empty(2 * step + K, dtype=torch.int8, device="cuda")
    x = xb.as_strided((M, K), (step, 1))
    x.copy_(_codes(M, K, K, 8))
    w = _codes(C, K, K, 9)
    ob = torch.empty(2 * (1 << 30) + C, dtype=BF16, device="cuda")
    out = ob.as_strided((M, C), (1 << 30, 1))
    sx, sw = _scales(M, 1), _scales(C, 2)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out, ws)
    _linear_close(out.contiguous(), x.contiguous(), sx, w, sw, None, BF16)


# ---------------------------------------------------------------------------
# rotary positions

def _rope_check(x, out, rope, pos, weight, eps, dtype):
    B, H, N, d = x.shape
    v = _f64(x.cpu())
    tol = 2.0 ** -18
    if weight is not None:
        full = weight.numel() != d
        axis = (1, 3) if full else (3,)
        v = v / np.sqrt((v * v).mean(axis, keepdims=True) + eps)
        v = v * (_f64(weight).reshape(1, H, 1, d) if full else _f64(weight))
    halves = rope.pairing == "halves"
    if pos is None:
        T, Hs, Ws = rope.grid
        n = np.arange(N)
        grid = np.stack([n // (Hs * Ws), n // Ws % Hs, n % Ws], -1).astype(float)
        ang = oracle.rope_angles(grid, rope.axes, rope.theta)
        ang[n >= T * Hs * Ws] = np.nan
        angles = [ang] * B
    else:
        p = pos.cpu().numpy()
        angles = [oracle.rope_angles(p if p.ndim == 2 else p[b], rope.axes, rope.theta) for b in range(B)]
    for b in range(B):
        ref = oracle.rope(v[b], angles[b], halves)
        if halves:
            size = np.abs(v[b][..., :d // 2]) + np.abs(v[b][..., d // 2:])
            size = np.concatenate([size, size], -1)
        else:
            size = np.repeat(np.abs(v[b][..., 0::2]) + np.abs(v[b][..., 1::2]), 2, -1)
        _close(out[b], ref, tol * size + _half(dtype) * 1.001 * np.abs(ref) + 1e-37)


ROPE = [  # B, H, N, d, axes, grid
    (1, 1, 1, 64, (32, 16, 16), (1, 1, 1)), (2, 3, 70, 64, (22, 20, 22), (3, 4, 5)), (1, 12, 131, 128, (44, 42, 42), (2, 8, 8)),
    (3, 40, 9, 128, (16, 56, 56), (1, 3, 3)), (1, 2, 33, 128, (0, 64, 64), (1, 4, 8)), (2, 1, 50, 64, (64, 0, 0), (50, 1, 1)),
    (1, 5, 260, 64, (2, 2, 60), (4, 5, 13)), (1, 24, 17, 128, (42, 44, 42), (5, 2, 3)), (2, 128, 3, 128, (42, 44, 42), (1, 1, 2)),
    (1, 7, 40, 128, (128, 0, 0), (40, 1, 1)),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("norm", ["none", "head", "full"])
@pytest.mark.parametrize("B,H,N,d,axes,grid", ROPE)
def test_rope(B, H, N, d, axes, grid, norm, pairing, dtype):
    g = _gen(N + H)
    rope = da.Rope(axes=axes, grid=grid, theta=10000.0 if d == 128 else 256.0, pairing=pairing)
    buf = torch.randn(B, N, 2, H, d, generator=g).to(dtype).cuda()
    x = buf[:, :, 1].permute(0, 2, 1, 3)
    weight = None if norm == "none" else (1 + 0.2 * torch.randn(d if norm == "head" else H * d, generator=g)).to(dtype).cuda()
    pos = torch.randint(-5000, 1 << 20, (B, N, 3), generator=g, dtype=torch.int32)
    pos[0, 0] = torch.tensor([(1 << 24) - 1, -(1 << 24), 0])
    for p in (None, pos.cuda(), pos[0].contiguous().cuda()):
        out = torch.full((B, H, N + 1, d), 9.0, dtype=dtype, device="cuda")
        before = buf.clone()
        da.da_rope(x, out[:, :, :N], rope, positions=p, weight=weight, eps=1e-5)
        assert torch.equal(buf, before) and (out[:, :, N] == 9).all()
        _rope_check(x, out[:, :, :N], rope, p, weight, 1e-5, dtype)
    # in place, on a slot of the buffer: the same bits, and the other slot untouched
    want = torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    da.da_rope(x, want, rope, weight=weight, eps=1e-5)
    da.da_rope(x, x, rope, weight=weight, eps=1e-5)
    assert torch.equal(x, want) and torch.equal(buf[:, :, 0], before[:, :, 0])


@pytest.mark.parametrize("B,N", [(300, 1), (65535, 1), (1, 1), (7, 33), (2, 4097)])
def test_rope_of_many_and_of_single_tokens(B, N):
    g = _gen(B)
    x = torch.randn(B, 2, N, 64, generator=g).to(BF16).cuda()
    out = torch.empty_like(x)
    pos = torch.randint(0, 5000, (N, 3), generator=g, dtype=torch.int32).cuda()
    rope = da.Rope((20, 22, 22), pairing="halves")
    da.da_rope(x, out, rope, positions=pos)
    _rope_check(x[:50], out[:50], rope, pos, None, 0, BF16)
    one = torch.empty_like(x[-1:])
    da.da_rope(x[-1:], one, rope, positions=pos)
    assert torch.equal(one, out[-1:])


def test_rope_at_the_ends_of_int32():
    """Positions of the whole int32 range against whole-number arithmetic of the turns in Python."""
    import math
    from fractions import Fraction
    x = torch.randn(1, 1, 4, 64, generator=_gen(3)).cuda()
    pos = torch.tensor([[-(1 << 31)] * 3, [(1 << 31) - 1] * 3, [123456789, -987654321, 1], [0, 0, 0]], dtype=torch.int32)
    out = torch.empty_like(x)
    # theta = 1: every pair of an axis turns by the position in radians
    da.da_rope(x, out, da.Rope((20, 22, 22), theta=1.0), positions=pos.cuda())
    two_pi = Fraction(628318530717958647692528676655900576839, 10 ** 38)
    ang = np.empty((4, 32))
    for n in range(4):
        for u, (lo, hi) in enumerate(((0, 10), (10, 21), (21, 32))):
            p = Fraction(int(pos[n, u]))
            ang[n, lo:hi] = float(p - two_pi * math.floor(p / two_pi))
    ref = oracle.rope(x.cpu(), ang, False)
    size = np.repeat(np.abs(_f64(x.cpu()))[..., 0::2] + np.abs(_f64(x.cpu()))[..., 1::2], 2, -1)
    _close(out, ref, 2.0 ** -18 * size)


def test_rope_far_positions_turn_as_the_formula_says():
    """Differences of positions: turning by p + q is turning by p, then by q; by -p undoes it."""
    g = _gen(1)
    x = torch.randn(1, 2, 64, 128, generator=g).cuda()
    rope = da.Rope(axes=(44, 42, 42))
    p, q = (torch.randint(0, 1 << 20, (64, 3), generator=g, dtype=torch.int32).cuda() for _ in range(2))
    once, first, twice, back = (torch.empty_like(x) for _ in range(4))
    da.da_rope(x, once, rope, positions=p + q)
    da.da_rope(x, first, rope, positions=p)
    da.da_rope(first, twice, rope, positions=q)
    da.da_rope(first, back, rope, positions=-p)
    size = x.abs().amax().item() * 2
    assert (once - twice).abs().max().item() <= 3 * 2.0 ** -18 * size and (back - x).abs().max().item() <= 2 * 2.0 ** -18 * size


def test_rope_leaves_text_rows_whatever_they_hold():
    x = torch.randn(1, 3, 12, 64, generator=_gen(2))
    x[0, 0, 10] = float("inf")
    x[0, 1, 11, 5] = float("nan")
    x[0, 2, 11, 7] = -0.0
    xc = x.cuda()
    out = torch.empty_like(xc)
    da.da_rope(xc, out, da.Rope(axes=(32, 16, 16), grid=(1, 2, 5), pairing="halves"))
    assert torch.equal(out[:, :, 10:].view(torch.int32), xc[:, :, 10:].view(torch.int32))
    assert torch.isfinite(out[:, :, :10]).all()


# ---------------------------------------------------------------------------
# streams, graphs, repetition

def _chain(seed, M=300, width=640, H=5, d=128):
    g = _gen(seed)
    s = dict(x=torch.randn(M, width, generator=g).to(BF16).cuda(), r=torch.randn(M, width, generator=g).to(BF16).cuda(),
             w=torch.ones(width).to(BF16).cuda(), wq=_codes(H * d, width, width, seed), ws_=_scales(H * d, seed).cuda(),
             q=torch.empty(M, width, dtype=torch.int8, device="cuda"), s=torch.empty(M, device="cuda"),
             sum=torch.empty(M, width, dtype=BF16, device="cuda"), h=torch.empty(1, H, M, d, dtype=BF16, device="cuda"),
             o=torch.empty(1, H, M, d, dtype=BF16, device="cuda"), q2=torch.empty(M, H * d, dtype=torch.int8, device="cuda"),
             s2=torch.empty(M, device="cuda"), ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    rope = da.Rope(axes=(44, 42, 42), grid=(3, 10, 10))

    def run():
        da.da_rms_norm_i8(s["x"], s["w"], s["q"], s["s"], residual=s["r"], sum_out=s["sum"])
        da.da_linear_i8(s["q"], s["s"], s["wq"], s["ws_"], s["h"], s["ws"])
        da.da_rope(s["h"], s["o"], rope)
        da.da_quantize_i8(s["o"], s["q2"], s["s2"])
    return s, run


def test_two_chains_at_once():
    """Two chains on two streams, issued in turns, without waiting: the bits of each alone."""
    chains = [_chain(seed, M=2000 + 300 * seed) for seed in (3, 4)]
    keys = ("sum", "q", "s", "h", "o", "q2", "s2")
    want = []
    for s, run in chains:
        run()
        torch.cuda.synchronize()
        want.append({k: s[k].clone() for k in keys})
        for k in keys:
            s[k].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(10):
        for stream, (s, run) in zip(streams, chains):
            with torch.cuda.stream(stream):
                run()
    torch.cuda.synchronize()
    for (s, _), w in zip(chains, want):
        assert all(torch.equal(s[k], w[k]) for k in keys) and da.da_device_status(s["ws"]) == 0


def test_same_bits_on_streams_and_in_graphs():
    s, run = _chain(1)
    run()
    torch.cuda.synchronize()
    want = {k: s[k].clone() for k in ("sum", "q", "s", "h", "o", "q2", "s2")}

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(s[k], v) for k, v in want.items())

    def clear():
        for k in want:
            s[k].zero_()
        torch.cuda.synchronize()
    clear()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    assert same()
    clear()
    t, run_t = _chain(2)                                        # another set captured into a graph of its own
    graphs = []
    for f in (run, run_t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graphs.append(graph)
    clear()
    other = torch.cuda.Stream()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    assert same()
    run_t()
    torch.cuda.synchronize()
    assert da.da_device_status(s["ws"]) == 0 and da.da_device_status(t["ws"]) == 0


# ---------------------------------------------------------------------------
# what the binding refuses by shape, type and stride

def _refused(code, f, *args, **kw):
    with pytest.raises(da.DAError) as e:
        f(*args, **kw)
    assert e.value.code == code, str(e.value)


def test_binding_refuses_shapes_types_and_strides():
    SHAPE, DTYPE, INVALID = 2, 3, 1
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(64, device="cuda")
    q, s, ws = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    b = x.to(BF16)
    _refused(DTYPE, da.da_rms_norm, x.half(), None, x)
    _refused(DTYPE, da.da_rms_norm, x, None, b)
    _refused(DTYPE, da.da_rms_norm, x, w.to(BF16), x)
    _refused(SHAPE, da.da_rms_norm, x, w[:63], x)
    _refused(SHAPE, da.da_rms_norm, x, w[None], x)
    _refused(SHAPE, da.da_rms_norm, x, None, x[:3])
    _refused(SHAPE, da.da_rms_norm, x, None, x.t())
    _refused(SHAPE, da.da_rms_norm, x[None], None, x[None])
    _refused(SHAPE, da.da_rms_norm, x, None, torch.empty(64, 4, device="cuda").t())
    _refused(SHAPE, da.da_rms_norm, x, None, x, residual=x[:, :63])
    _refused(INVALID, da.da_rms_norm, x, None, x.cpu())
    _refused(INVALID, da.da_rms_norm, x, None, torch.empty_like(x), sum_out=x)      # a sum without a residual
    _refused(INVALID, da.da_rms_norm, x[:0], None, x[:0])
    _refused(DTYPE, da.da_rms_norm_i8, x, None, x, s)
    _refused(SHAPE, da.da_rms_norm_i8, x, None, q, s[:3])
    _refused(DTYPE, da.da_quantize_i8, q, q, s)
    _refused(SHAPE, da.da_quantize_i8, x.view(2, 2, 64), q, s)
    _refused(SHAPE, da.da_quantize_i8, x.view(1, 2, 2, 64), q, s)
    _refused(SHAPE, da.da_linear_i8, q, s, q, s, x, ws)                             # out is [4, 64], not [4, 4]
    _refused(DTYPE, da.da_linear_i8, q, s, q, s, torch.zeros(4, 4, dtype=torch.int32, device="cuda"), ws)
    _refused(SHAPE, da.da_linear_i8, q, s, q, s, torch.zeros(1, 2, 4, 4, device="cuda"), ws)
    _refused(9, da.da_linear_i8, q, s, q, s, torch.zeros(4, 4, device="cuda"), ws[:255])
    _refused(SHAPE, da.da_linear_i8, q, s, q, s, torch.zeros(4, 4, device="cuda"), ws.repeat(2)[::2])
    h, rope = torch.zeros(1, 1, 4, 64, device="cuda"), da.Rope((32, 16, 16), (1, 2, 2))
    o = torch.empty_like(h)
    _refused(SHAPE, da.da_rope, h[0], o[0], rope)
    _refused(SHAPE, da.da_rope, h, o[:, :, :3], rope)
    _refused(DTYPE, da.da_rope, h, o.to(BF16), rope)
    _refused(DTYPE, da.da_rope, h, o, rope, positions=torch.zeros(4, 3, dtype=torch.int64, device="cuda"))
    _refused(SHAPE, da.da_rope, h, o, rope, positions=torch.zeros(3, 3, dtype=torch.int32, device="cuda"))
    _refused(SHAPE, da.da_rope, h, o, rope, weight=torch.zeros(65, device="cuda"))
    _refused(SHAPE, da.da_rope, h, o, da.Rope((32, 16, 16)))                        # neither a grid nor positions
    with pytest.raises(TypeError):
        da.da_rms_norm(x, None, torch.empty_like(x), eps="small")
    with pytest.raises(TypeError):
        da.da_rope(h, o, da.Rope((32, 16, 16), (1, 2, 2), theta="large"))


def test_stream_arguments():
    """A stream object, its handle and the current stream are the same to a call."""
    x = torch.randn(64, 256, generator=_gen(1)).cuda()
    want, out = torch.empty_like(x), torch.empty_like(x)
    da.da_rms_norm(x, None, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        da.da_rms_norm(x, None, out, stream=stream)
        side.synchronize()
        assert torch.equal(out, want)
    with pytest.raises(TypeError):
        da.da_rms_norm(x, None, out, stream="side")
