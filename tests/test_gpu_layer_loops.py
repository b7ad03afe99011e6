"""The loops of the layer operators' kernels, turned often: blocks of the rotary kernel that take many tokens one after another,
CTAs of the product that take many tiles.  Small shapes give every block one token or tile, and then neither a ring's second
filling, nor a barrier's second phase, nor an accumulator's second use is reached.

Each case states what it is meant to reach, and a restatement of the library's launch rules checks that it does.  Tolerances
are those of test_gpu_layer.py.
"""
import numpy as np
import pytest
import torch

import block_sparse_cluster_b200 as da
from tests.test_gpu_layer import BF16, F32, _codes, _gen, _linear_close, _rope_check, _scales

pytestmark = pytest.mark.gpu

SMS = 148


# ---------------------------------------------------------------------------
# rotary positions

def _turns(B, H, N, d, norm, dtype):
    """(tokens that a group of threads takes, groups of a block), as the library chooses them."""
    per_head = d // 2 * dtype.itemsize // 16
    heads = H if norm == "full" else min(H, 1024 // per_head)
    units = heads * per_head
    if units <= (128 if norm == "none" else 64):
        group = per_head
        while group < units and group < 32:
            group *= 2
        upt, threads = (units + 31) // 32, 128
    else:
        upt = 1 if units <= (256 if norm == "full" else 512) else 2 if units <= 1024 else 4
        threads = group = ((units + upt - 1) // upt + 31) // 32 * 32
    groups, turns = threads // group, 1
    blocks = SMS * (8 if upt >= 2 and threads > 128 else 16)
    while turns < (16 if upt >= 2 and norm == "full" else 8) and groups * turns * 2 <= 32 and B * N // (groups * turns * 2) >= blocks:
        turns *= 2
    return turns, groups


@pytest.mark.parametrize("B,H,N,d,norm,dtype,pairing,turns,groups", [
    (1, 12, 19003, 128, "full", BF16, "adjacent", 8, 1), (1, 40, 19003, 128, "full", BF16, "halves", 16, 1),
    (1, 40, 19003, 128, "none", BF16, "halves", 8, 1), (2, 12, 9507, 128, "head", BF16, "adjacent", 8, 1),
    (1, 8, 76001, 128, "head", BF16, "halves", 8, 4), (1, 2, 76001, 64, "none", BF16, "adjacent", 2, 16),
    (1, 4, 76003, 128, "full", BF16, "adjacent", 8, 4), (1, 12, 19001, 128, "full", F32, "halves", 8, 1),
    (1, 3, 38001, 64, "head", F32, "adjacent", 4, 4), (1, 70, 9601, 128, "full", F32, "adjacent", 8, 1),
])
def test_rope_of_long_runs(B, H, N, d, norm, dtype, pairing, turns, groups):
    assert _turns(B, H, N, d, norm, dtype) == (turns, groups) and (turns > 3 or groups > 4) and N % (turns * groups)
    g = _gen(N + H)
    rope = da.Rope(axes=(44, 42, 42) if d == 128 else (20, 22, 22), pairing=pairing)
    buf = torch.randn(B, N, 2, H, d, generator=g).to(dtype).cuda()
    x = buf[:, :, 1].permute(0, 2, 1, 3)
    weight = None if norm == "none" else (1 + 0.2 * torch.randn(d if norm == "head" else H * d, generator=g)).to(dtype).cuda()
    pos = torch.randint(-5000, 1 << 20, (B, N, 3), generator=g, dtype=torch.int32).cuda()
    out = torch.full((B, H, N + 1, d), 9.0, dtype=dtype, device="cuda")
    da.da_rope(x, out[:, :, :N], rope, positions=pos, weight=weight, eps=1e-5)
    assert (out[:, :, N] == 9).all()
    # the head, the tail and the borders of runs against the oracle
    run = turns * groups
    borders = torch.randint(1, N // run, (20,), generator=g) * run
    some = torch.cat([torch.arange(2 * run), N - 1 - torch.arange(2 * run), borders - 1, borders]).unique()
    _rope_check(x[:, :, some.cuda()], out[:, :, :N][:, :, some.cuda()], rope, pos[:, some.cuda()].contiguous(), weight, 1e-5, dtype)
    # the whole against calls short enough for single turns: the same bits
    for lo in range(0, N, 1000):
        hi = min(lo + 1000, N)
        assert _turns(B, H, hi - lo, d, norm, dtype)[0] == 1
        part = torch.empty(B, H, hi - lo, d, dtype=dtype, device="cuda")
        da.da_rope(x[:, :, lo:hi], part, rope, positions=pos[:, lo:hi].contiguous(), weight=weight, eps=1e-5)
        assert torch.equal(part, out[:, :, lo:hi]), lo
    # by the grid, with tokens behind it; then in place, on the buffer's slot
    grid = da.Rope(axes=rope.axes, grid=(9, 31, (N - 200) // 279), pairing=pairing)
    cells = 9 * 31 * ((N - 200) // 279)
    n = torch.arange(cells, dtype=torch.int32)
    where = torch.stack([n // (31 * grid.grid[2]), n // grid.grid[2] % 31, n % grid.grid[2]], -1).contiguous().cuda()
    want = torch.empty(B, H, N, d, dtype=dtype, device="cuda")
    da.da_rope(x, want, grid, weight=weight, eps=1e-5)
    turned = torch.empty(B, H, cells, d, dtype=dtype, device="cuda")
    da.da_rope(x[:, :, :cells], turned, rope, positions=where, weight=weight, eps=1e-5)
    assert torch.equal(want[:, :, :cells], turned)
    if norm == "none":
        assert torch.equal(want[:, :, cells:], x[:, :, cells:])
    before = buf[:, :, 0].clone()
    da.da_rope(x, x, grid, weight=weight, eps=1e-5)
    assert torch.equal(x, want) and torch.equal(buf[:, :, 0], before)


# ---------------------------------------------------------------------------
# product

def _tiles(M, N, K):
    """(CTA pairs, columns of a tile, most tiles of a pair or a CTA), as the library chooses them."""
    up = lambda a, b: -(-a // b)
    k, best, least = up(K, 32), None, 0
    for n in range(256, 159, -32):
        clocks = up(up(M, 256) * up(N, n), SMS // 2) * (n // 2 * k + 2000)
        if best is None or clocks < least:
            least, best = clocks, (True, n)
    for n in range(16, 257, 16):
        clocks = up(up(M, 128) * up(N, n), SMS) * (max(n // 2, 32 + n // 4) * k * 5 // 4 + 2000)
        if clocks < least or (clocks == least and not best[0]):
            least, best = clocks, (False, n)
    pair, n = best
    return pair, n, up(up(M, 256 if pair else 128) * up(N, n), SMS // 2 if pair else SMS)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K,pair,n,tiles", [
    (9001, 2901, 144, True, 256, 6), (6000, 6016, 128, True, 256, 8), (8192, 4096, 272, True, 256, 7),
    (100000, 8, 64, False, 16, 6), (100000, 24, 700, False, 32, 6), (15641, 1032, 362, False, 176, 5),
])
def test_linear_of_many_tiles_a_cta(M, C, K, pair, n, tiles, dtype):
    """Both accumulators used again and again, by pairs and by single CTAs, ragged on every side; heads where they fit."""
    assert _tiles(M, C, K) == (pair, n, tiles)
    x, w = _codes(M, K, -(-K // 16) * 16, 1), _codes(C, K, -(-K // 16) * 16, 2)
    sx, sw, bias = _scales(M, 3), _scales(C, 4), torch.randn(C, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for gap in (8, 3):                                           # output rows on 16 bytes, and anywhere
        out = torch.full((M + 1, C + gap), 7.0, dtype=dtype, device="cuda")
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:M, :C], ws, bias=bias.cuda())
        assert da.da_device_status(ws) == 0
        _linear_close(out[:M, :C], x, sx, w, sw, bias, dtype)
        assert (out[M:] == 7).all() and (out[:, C:] == 7).all()
    if C % 128 == 0:
        heads = torch.full((2, C // 128, M // 2, 128), 7.0, dtype=dtype, device="cuda")
        da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), heads, ws, bias=bias.cuda())
        assert torch.equal(heads.permute(0, 2, 1, 3).reshape(M, C), out[:M, :C]) and da.da_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K", [(5, 60000, 256), (60, 100000, 256), (7, 120000, 544)])
def test_linear_of_few_rows_and_many_tiles(M, C, K, dtype):
    """A tile of fewer than 128 rows of x, and more tiles than processors."""
    pair, n, tiles = _tiles(M, C, K)
    assert not pair and tiles >= 2
    x, w = _codes(M, K, K, 1), _codes(C, K, K, 2)
    sx, sw = _scales(M, 3), _scales(C, 4)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 1, C + 8), 7.0, dtype=dtype, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:M, :C], ws)
    assert da.da_device_status(ws) == 0
    _linear_close(out[:M, :C], x, sx, w, sw, None, dtype)
    assert (out[M:] == 7).all() and (out[:, C:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,C,K,n", [(777, 1537, 1001, 64), (1300, 1000, 515, 64), (640, 2000, 130, 64), (2000, 3001, 260 + 7, 128), (200, 1300, 999, 32)])
def test_linear_off_16_bytes_in_tiles_of_every_width(M, C, K, n, dtype):
    """Rows packed at a depth that is no multiple of 16; the tile is 128 columns, or 64 or 32 where that fills the GPU."""
    rows = -(-M // 128)
    assert K % 16 and n == (128 if rows * -(-C // 128) >= SMS else 64 if rows * -(-C // 64) >= SMS else 32)
    x, w = _codes(M, K, K, 1), _codes(C, K, K, 2)
    sx, sw, bias = _scales(M, 3), _scales(C, 4), torch.randn(C, generator=_gen(6))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 1, C + 3), 7.0, dtype=dtype, device="cuda")
    da.da_linear_i8(x, sx.cuda(), w, sw.cuda(), out[:M, :C], ws, bias=bias.cuda())
    assert da.da_device_status(ws) == 0
    _linear_close(out[:M, :C], x, sx, w, sw, bias, dtype)
    assert (out[M:] == 7).all() and (out[:, C:] == 7).all()


@pytest.mark.parametrize("M,C", [(6, 40), (129, 40), (300, 520), (2000, 2100)])
@pytest.mark.parametrize("pitch", [131072, 131071])
def test_linear_of_the_deepest_sums(pitch, M, C):
    """K = 131071 with every code -128, the largest sum there is, on the tensor cores: tile loads, and rows off 16 bytes."""
    K = 131071
    x = torch.full((M, pitch), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((C, pitch), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1], x[3] = 127, 127
    out = torch.empty(M, C, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    da.da_linear_i8(x, torch.ones(M).cuda(), w, torch.ones(C).cuda(), out, ws)
    assert da.da_device_status(ws) == 0
    a, b = np.full(M, -128.0), np.full(C, -128.0)
    a[3], b[1] = 127, 127
    want = np.outer(a, b) * K                                    # whole numbers, rounded once to fp32
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))
