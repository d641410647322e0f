"""Every kernel variant of the block-scaled FP8 operators at sizes that reach it.

`dense_shape` and `experts_shape` repeat the library's choice of a product's tile on the
host; each case names the variant it is meant for, and the host test fails where the
choice has moved away from it.  Products use whole codes and scales of 1/2, 1 and 2, so
the results are exact; operands' padding holds NaN codes and the results' stays untouched.
"""

import ctypes

import numpy as np
import pytest
import torch

from .test_fp8_block_abi import NormArgs, _lib
from .test_gpu_fp8_block import (DTYPES, NORM, U, check_product, check_quantized, check_rounded, gen,
                                 plain_permute, quantized_pair, step_of)

gpu = pytest.mark.gpu


def up(a, b):
    return -(-a // b)


def few_rows(items):
    return "16x16 two waves" if items > 512 else "16x16 eight waves"


def fits(bm, bn, N, tiles, grouped):
    """Whether a launch of this tile stays within 2^20 workgroups."""
    per = 1
    if grouped and tiles > 128:
        per = 16 if bm > 64 and up(N, bn) % 4 == 0 else 32 if bm > 64 else 8
    return up(tiles, per) * per * up(N, bn) <= 1 << 20


def dense_shape(M, N, K):
    def count(bm, bn):
        return up(M, bm) * up(N, bn)
    if M <= 16 or (M <= 128 and count(16, 16) * 32 * K <= 48e6):
        return few_rows(count(16, 16))
    if K <= 1024 and count(64, 128) <= 768:
        return "64x128"
    for bm, bn, name in ((64, 32, "64x32 x6"), (64, 64, "64x64 x4"), (64, 128, "64x128 x3"),
                         (128, 128, "128x128 x2")):
        if count(bm, bn) <= 256:
            return name
    time = {256: up(count(256, 256), 256), 192: 0.79 * up(count(192, 256), 256),
            128: 0.57 * up(count(128, 256), 256)}
    bm = 128 if time[128] < min(time[192], time[256]) else 192 if time[192] < time[256] else 256
    return f"{bm}x256" if fits(bm, 256, N, up(M, bm), False) else few_rows(count(16, 16))


def experts_shape(M, E, N, max_tiles, block_m):
    tiles = min(max_tiles, E + M // 64) * up(N, 128)
    if M // E > 128:
        bm, bn, name = 192, 256, "192x256"
    elif M // E > 32:
        bm, bn, name = 128, 256, "128x256"
    elif tiles >= 400:
        bm, bn, name = 64, 128, "64x128"
    elif M > 32:
        bm, bn, name = 64, 128, "64x128 x3"
    else:
        return few_rows(max_tiles * up(block_m, 16) * up(N, 16))
    if fits(bm, bn, N, max_tiles * up(block_m, bm), True):
        return name
    return few_rows(max_tiles * up(block_m, 16) * up(N, 16))


# Row lengths: whole blocks and a short last one, below, at and above the variants' counts
# of K groups and of blocks in flight; where reachable, rows shorter than a block.
DENSE = {
    "16x16 eight waves": [(3, 129, 16), (17, 500, 112), (33, 119, 4096), (16, 100, 4240), (5, 77, 5136),
                          (1, 50, 6160), (9, 130, 3200), (128, 31, 1040)],
    "16x16 two waves": [(3, 9001, 400), (1, 9001, 112), (2, 8300, 1280), (1, 8209, 1536), (5, 8200, 1792),
                        (16, 8301, 1664), (1, 9001, 2064), (17, 4515, 1168), (7, 8250, 128), (40, 3001, 1040)],
    "64x128": [(153, 101, 112), (130, 500, 912), (1030, 260, 16), (257, 513, 272), (2001, 1003, 1024)],
    "64x32 x6": [(153, 101, 1168), (200, 700, 2064), (131, 333, 1040), (300, 999, 1664), (129, 65, 1152)],
    "64x64 x4": [(66, 8185, 1168), (1001, 701, 1040), (1000, 700, 1152), (257, 3001, 1296), (999, 701, 2064)],
    "64x128 x3": [(130, 9001, 1168), (1500, 1203, 1040), (1501, 1200, 1280), (1003, 1801, 2000)],
    "128x128 x2": [(5534, 257, 1168), (1500, 2001, 1040), (1501, 2000, 1152), (1999, 1999, 1296)],
    "128x256": [(5413, 641, 1168), (2501, 2503, 1040), (4873, 1163, 112), (4873, 1163, 16), (2501, 2501, 1280)],
    "192x256": [(5404, 1285, 1168), (3001, 3101, 1152), (5404, 1285, 112), (5405, 1283, 48), (2049, 4101, 144)],
    "256x256": [(5380, 2053, 1168), (5381, 2051, 1040), (5380, 2053, 112), (5383, 2055, 16), (5381, 2050, 272),
                (5380, 2053, 1280)],
}
DENSE_CASES = [(shape, *c) for shape, cases in DENSE.items() for c in cases]

# rows, experts, N, entry rows, what is expected
EXPERTS = [
    (9, 5, 333, 16, "16x16 eight waves"), (30, 3, 200, 16, "16x16 eight waves"),
    (6, 8, 2001, 16, "16x16 two waves"), (32, 4, 1500, 128, "16x16 two waves"),
    (300, 40, 130, 32, "64x128 x3"), (40, 3, 515, 16, "64x128 x3"),
    (350, 60, 1030, 16, "64x128"), (900, 30, 1701, 128, "64x128"),
    (700, 10, 530, 64, "128x256"), (1500, 20, 900, 16, "128x256"),
    (700, 3, 530, 128, "192x256"), (2500, 4, 1030, 16, "192x256")]


def routed(rows, E, block_m):
    """Expert ids, uneven, one expert without rows, and the length of their tile list."""
    rng = np.random.default_rng(rows)
    ids = rng.choice(E, rows, p=np.arange(1, E + 1) / (E * (E + 1) / 2))
    ids[ids == 1] = E - 1
    return ids, sum(up(int(n), block_m) for n in np.bincount(ids, minlength=E)) + 3


def test_cases_reach_the_variants_they_name():
    for shape, M, N, K in DENSE_CASES:
        assert dense_shape(M, N, K) == shape, (M, N, K)
    for rows, E, N, block_m, shape in EXPERTS:
        _, max_tiles = routed(rows, E, block_m)
        assert experts_shape(rows, E, N, max_tiles, block_m) == shape, (rows, E, N)
    assert len({c[4] for c in EXPERTS}) == 6


@gpu
@pytest.mark.parametrize("shape,M,N,K", DENSE_CASES)
def test_dense_variants(gpu_lib, shape, M, N, K):
    dt = torch.float16 if (M + N) % 2 else torch.bfloat16
    a, sa, w, sw = quantized_pair(gen(M + N + K), M, N, K, lda=K + 16, ldw=K + 32, whole=True)
    room = torch.full((M, N + 3), 7.0, dtype=dt, device="cuda")
    out = gpu_lib.fp8_block_linear(a, sa, w, sw, out=room[:, :N])
    rows = torch.arange(M) if M < 300 else torch.cat([torch.arange(0, M - 80, 31), torch.arange(M - 80, M)])
    rows = rows.cuda()
    check_product(out[rows], a[rows], sa[rows], w, sw, shape, True)
    if M >= 300:                                     # every row, of some columns
        for b in sorted({0, (N // 2) // 128, (N - 1) // 128}):
            c = torch.arange(128 * b, min(N, 128 * b + 128), 9, device="cuda")
            check_product(out[:, c], a, sa, w[c], sw[b:b + 1], shape + " columns", True)
    assert bool((room[:, N:] == 7.0).all())


@gpu
@pytest.mark.parametrize("rows,E,N,block_m,shape", EXPERTS)
def test_expert_variants(gpu_lib, rows, E, N, block_m, shape):
    ids, _ = routed(rows, E, block_m)
    perm, offsets, order = plain_permute(ids, E, block_m)
    src = torch.from_numpy(order).cuda()
    # one to three blocks behind a wave's four in flight as well
    for K in (16, 112, 128, 400, 1168) + ((1280, 1536, 1792) if "wave" in shape else ()):
        a, sa, w, sw = quantized_pair(gen(K), rows, N, K, lda=K + 16, ldw=K + 16, E=E, whole=True)
        room = torch.full((rows, N + 5), 7.0, dtype=torch.float16, device="cuda")
        out = gpu_lib.fp8_block_grouped_gemm(a, sa, w, sw, perm, block_m, out=room[:, :N],
                                             a_row_gather=perm["sorted_pairs"])
        for e in range(E):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            if hi > lo:
                at = src[lo:hi]
                check_product(out[lo:hi], a[at], sa[at], w[e], sw[e], f"{shape} K={K} expert {e}", True)
        assert bool((room[:, N:] == 7.0).all())


@gpu
@pytest.mark.parametrize("rows,E", [(20, 5), (300, 4)])
def test_a_tile_list_longer_than_a_grid(gpu_lib, rows, E):
    """Mostly unused entries: more workgroups than one launch takes, so the 16x16 kernel
    steps over the list."""
    N, K, block_m = 4100, 400, 128
    ids, _ = routed(rows, E, block_m)
    perm, offsets, order = plain_permute(ids, E, block_m)
    room = torch.full((70000, 2), 10 ** 6, dtype=torch.int32, device="cuda")
    room[:perm["tiles"].shape[0]] = perm["tiles"]
    perm = dict(perm, tiles=room, max_tiles=len(room))
    assert experts_shape(rows, E, N, len(room), block_m).startswith("16x16")
    a, sa, w, sw = quantized_pair(gen(rows), rows, N, K, E=E, whole=True)
    out = gpu_lib.fp8_block_grouped_gemm(a, sa, w, sw, perm, block_m, a_row_gather=perm["sorted_pairs"])
    src = torch.from_numpy(order).cuda()
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            check_product(out[lo:hi], a[src[lo:hi]], sa[src[lo:hi]], w[e], sw[e], f"expert {e}", True)


# ------------------------------------------------------------------ norm

def norm_inputs(M, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((M, K), generator=g, device="cuda") *
         torch.exp(torch.randn((M, 1), generator=g, device="cuda"))).to(DTYPES[dtype])
    r = (3 * torch.randn((M, K), generator=g, device="cuda")).to(DTYPES[dtype])
    w = (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(DTYPES[dtype])
    return x, r, w


@gpu
@pytest.mark.parametrize("M,K,dtype", [(300, 7168, "bf16"), (260, 4104, "f16"), (257, 8191, "bf16"),
                                       (270, 5000, "f32"), (300, 4095, "bf16"), (259, 16384, "f32")])
def test_norm_of_prefill_rows(gpu_lib, M, K, dtype):
    """More than 256 rows of 4097 to 8192 columns take two pieces a thread."""
    x, r, w = norm_inputs(M, K, dtype, K)
    y = torch.empty_like(x)
    c, s, ro = gpu_lib.rms_norm_fp8(x, w, eps=1e-5, residual=r, y=y)
    assert torch.equal(ro, (x.float() + r.float()).to(x.dtype))
    v = (x.double() + r.double()).cpu().numpy()
    ref = v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-5) * w.double().cpu().numpy()
    check_quantized(c, s, ref, NORM, "norm")
    check_rounded(y, ref, NORM * np.abs(ref), "y")


@gpu
@pytest.mark.parametrize("M,K,dtype", [(5000, 7168, "bf16"), (2600, 7168, "f32"), (70000, 512, "bf16"),
                                       (40000, 1000, "f16"), (17000, 2048, "bf16"), (9000, 4096, "f16"),
                                       (2200, 16384, "bf16"), (2200, 16384, "f32")])
def test_norm_streams_large_results_as_it_writes_small_ones(gpu_lib, M, K, dtype):
    """Results above 64 MB go past the caches, residual_out in place among them: the same
    bits as in pieces that do not (and that take the same threads a row)."""
    x, r, w = norm_inputs(M, K, dtype, M)
    assert M * K * x.element_size() > 64 << 20
    keep, y = r.clone(), torch.empty_like(x)
    c, s, ro = gpu_lib.rms_norm_fp8(x, w, residual=r, residual_out=r, y=y)
    assert ro is r
    for lo in list(range(0, M, 1000))[:-1] + [M - 1000]:
        at = slice(lo, lo + 1000)
        assert 1000 * K * x.element_size() <= 64 << 20
        py = torch.empty_like(x[at])
        pc, ps, pr = gpu_lib.rms_norm_fp8(x[at], w, residual=keep[at], y=py)
        assert torch.equal(c[at], pc) and torch.equal(s[at], ps), lo
        assert torch.equal(ro[at], pr) and torch.equal(y[at], py), lo


@gpu
@pytest.mark.parametrize("K", [24, 9, 1000])
def test_norm_of_more_rows_than_a_grid(gpu_lib, K):
    """2^20 workgroups at most: the rows above are their second ones."""
    M = 2 ** 20 + 300
    x, r, w = norm_inputs(M, K, "bf16", K)
    c, s, ro = gpu_lib.rms_norm_fp8(x, w, residual=r)
    assert torch.equal(ro, (x.float() + r.float()).bfloat16())
    for lo in (0, 2 ** 19, 2 ** 20 - 300, 2 ** 20):
        at = slice(lo, lo + 300)
        pc, ps, _ = gpu_lib.rms_norm_fp8(x[at].clone(), w, residual=r[at].clone())
        assert torch.equal(c[at], pc) and torch.equal(s[at], ps), lo


@gpu
@pytest.mark.parametrize("K", [640, 7168, 20480])
def test_norm_without_codes(gpu_lib, K):
    """The C call writes y and residual_out alone where codes and scales are null."""
    M = 5
    x, r, w = norm_inputs(M, K, "bf16", 3)
    want = torch.empty_like(x)
    _, _, want_r = gpu_lib.rms_norm_fp8(x, w, residual=r, y=want)
    y, ro = torch.empty_like(x), torch.empty_like(x)
    args = NormArgs(dtype=0, M=M, K=K, eps=1e-6, x=x.data_ptr(), ldx=K, residual=r.data_ptr(), ldr=K,
                    weight=w.data_ptr(), residual_out=ro.data_ptr(), ldro=K, y_out=y.data_ptr(), ldy=K)
    assert _lib().rms_norm_fp8(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y, want) and torch.equal(ro, want_r)


@gpu
@pytest.mark.parametrize("M,K,dtype", [(300, 7168, "bf16"), (1000, 2048, "f16"), (1000, 2048, "f32"),
                                       (100, 20480, "bf16")])
def test_norm_codes_next_to_the_middle(gpu_lib, M, K, dtype):
    """The codes come from the exact products v*w over their block's largest, with one
    float32 rounding of the quotient (u relative, and a 2^-16th of it for the rest): only a
    quotient that close to the middle of two codes may get the other one.  Float32
    arithmetic step by step is off by several times that."""
    x, r, w = norm_inputs(M, K, dtype, 7)
    c, _, _ = gpu_lib.rms_norm_fp8(x, w, residual=r)
    v = (x.float() + r.float()).double()                  # v is float32
    p = (v * w.double()).view(M, K // 128, 128)           # 48 bits: exact in float64
    q = (p * 448 / p.abs().amax(2, keepdim=True)).view(M, K).cpu().numpy()
    got = c.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    step = step_of(np.minimum(np.abs(q), 448))
    assert np.all(np.abs(got - q) <= 0.5 * step + U * (1 + 2.0 ** -16) * np.abs(q))


@gpu
def test_e4m3_middles_and_their_neighbours(gpu_lib):
    """Every middle between two codes, exactly and one float32 to either side, of both
    signs, in blocks whose scale is 1 (the first value is 448): middles go to the even code."""
    code = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    mid = ((code[1:].astype(np.float64) + code[:-1]) / 2).astype(np.float32)     # exact
    near = np.concatenate([code, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(500))])
    near = np.concatenate([near, -near])
    near = np.concatenate([near, np.zeros(-len(near) % 127, np.float32)]).reshape(-1, 127)
    w = torch.from_numpy(np.concatenate([np.full((len(near), 1), 448, np.float32), near], 1)).reshape(-1)
    x = torch.ones((1, w.numel()), device="cuda")
    c, s, _ = gpu_lib.rms_norm_fp8(x, w.cuda(), eps=0.0)
    assert torch.all(s == 1)
    q = w.double().numpy()
    step = step_of(q)
    want = np.rint(q / step) * step                       # rint: ties to even
    got = c[0].view(torch.float8_e4m3fn).float().double().cpu().numpy()
    assert np.array_equal(got, want)
