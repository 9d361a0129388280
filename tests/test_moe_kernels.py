"""Every kernel of the norm and of the experts' products that the library holds, by name: a call that takes it; products
with several stages of K, rows that end anywhere inside a tile, columns past the last workgroup's and pairs without an
expert."""
import functools
import re
import shutil
import subprocess

import numpy as np
import pytest

import moe_ref as ref
from test_gpu_moe import _dev, _norm_check, _rows, _say, env          # noqa: F401  (env: the fixture)

CODE = {"q4_0": 0, "q8_0": 1, "q2_k": 2, "q4_k": 3, "q6_k": 4, "q4_1": 5, "q5_0": 6, "q5_1": 7}
K_QUANTS, ON_GRID, ODD = ("q2_k", "q4_k", "q6_k"), ("q4_1", "q5_1"), ("q4_0", "q8_0", "q5_0")
BLOCKS32 = ODD + ON_GRID


def _cases():
    """(kernel, format, T, top, E, N, K, a row for each pair).  Workgroups counts, which choose a kernel, are those of
    blocks of 128 weight rows: one for every expert in use and one for every 16 (32) pairs."""
    few = {8: (6, 12), 16: (8, 15, 24), 32: (31, 60), 64: (63, 128, 140, 131)}         # blocks of a row
    for fmt in BLOCKS32:
        c = CODE[fmt]
        for lanes, blocks in few.items():
            for nb in blocks:
                paired = nb % 2 == 0
                units = nb // 2 if paired else nb
                lanes = next((n for n in (8, 16, 32) if units <= n), 64)
                yield (f"k_experts_few<{c}, {str(paired).lower()}, {lanes}, {1 if lanes == 64 else 2}>", fmt, 1, 3, 5, 37,
                       32 * nb, nb % 4 == 0)
        yield f"k_experts_few<{c}, false, 8, 2>", fmt, 1, 3, 5, 37, 32 * 7, False
        for rows, workgroup, T, top, E, N in ((16, "1, 2", 40, 2, 64, 776), (16, "2, 2", 20, 4, 16, 904),
                                              (16, "4, 2", 33, 2, 16, 40), (32, "1, 2", 200, 2, 16, 1800),
                                              (32, "2, 2", 100, 2, 8, 1400), (32, "4, 2", 90, 1, 2, 200),
                                              (32, "2, 2", 2200, 2, 7, 72)):           # a plan's 128 rows in parts of 32
            for K in (768, 1280):
                yield f"k_experts_stream<qmm::Blocks32<{c}, (qmm::Rows)0>, {rows}, {workgroup}>", fmt, T, top, E, N, K, K > 1000
        for rows, T, top, E, N in ((16, 33, 2, 16, 40), (32, 90, 1, 2, 200)):
            # an even number of blocks, and an odd one where no lead is needed or tiles of 32 rows are few
            blocks = (18, 30) if fmt in ODD and rows == 16 else (18, 31)
            for nb in blocks:
                yield f"k_experts_stream<qmm::Blocks32<{c}, (qmm::Rows)1>, {rows}, 4, 2>", fmt, T, top, E, N, 32 * nb, nb < 20
        if fmt in ODD:
            for rows, workgroup, T, top, E, N in ((16, "1, 2", 40, 2, 64, 776), (16, "2, 2", 20, 4, 16, 904),
                                                  (16, "4, 2", 33, 2, 16, 40), (32, "1, 4", 200, 2, 16, 1800)):
                for nb in (17, 31):
                    yield (f"k_experts_stream<qmm::Blocks32<{c}, (qmm::Rows)2>, {rows}, {workgroup}>", fmt, T, top, E, N,
                           32 * nb, nb < 20)
        yield f"k_experts_matmul<{c}, true>", fmt, 200, 2, 16, 1800, 32 * 22, False
        yield f"k_experts_matmul<{c}, false>", fmt, 2100, 2, 8, 904, 32 * 22, False
        yield f"k_experts_matmul<{c}, false>", fmt, 2100, 2, 8, 904, 32 * 23, True
    for fmt in K_QUANTS:
        c = CODE[fmt]
        for lanes, blocks in ((8, (2,)), (16, (3, 4)), (32, (5, 8)), (64, (9, 16, 17, 33))):
            for nb in blocks:
                yield f"k_experts_few<{c}, false, {lanes}, {1 if lanes == 64 else 2}>", fmt, 1, 3, 5, 37, 256 * nb, nb % 2 == 0
        for rows, workgroup, T, top, E, N in ((16, "1, 4", 40, 2, 64, 1032), (16, "1, 2", 40, 2, 64, 776),
                                              (16, "2, 2", 20, 4, 16, 904), (16, "4, 2", 33, 2, 16, 40),
                                              (32, "1, 4", 200, 2, 16, 2312), (32, "1, 2", 200, 2, 16, 1800),
                                              (32, "2, 2", 100, 2, 8, 1400), (32, "4, 2", 90, 1, 2, 200),
                                              (32, "2, 2", 2200, 2, 7, 72),            # a plan's 128 rows in parts of 32
                                              (64, "1, 4", 2100, 2, 16, 904)):         # and of 64
            for K in (768, 1024) if rows == 64 else (768, 1280):
                yield f"k_experts_stream<qmm::SuperBlocks<{c}>, {rows}, {workgroup}>", fmt, T, top, E, N, K, K == 768
        # many rows an expert, and so few pairs that the plan's tiles have 32
        yield f"k_experts_stream<qmm::SuperBlocks<{c}>, 32, 1, 4>", fmt, 1000, 2, 4, 1048, 768, False
    for K in (768, 1024):
        yield "k_experts_matmul_k<4>", "q6_k", 1700, 3, 8, 400, K, K == 768


CASES = list(_cases())


def _norms():
    """(kernel, dtype, format, T, K): pieces of 16 bytes a thread, for many rows (up to four on 256 threads, then more
    threads) and for few (a thread a piece, up to 1024)."""
    for r, (dtype, v) in enumerate((("f32", 4), ("f16", 8), ("bf16", 8))):
        for f, fmt in enumerate(("q8_0", "q8_k")):
            for T, pieces, held in ((300, 256, 1), (300, 512, 2), (300, 704, 4), (300, 1024, 4), (300, 1408, 4),
                                    (300, 2816, 4), (300, 4160, 0), (3, 1024, 1), (3, 1088, 2), (3, 2816, 4), (3, 4160, 0)):
                yield f"k_rms_norm<{r}, {f}, {v}, {held}>", dtype, fmt, T, v * pieces


NORMS = list(_norms())


def test_every_kernel_is_listed():
    """The library's own symbols against the cases."""
    import matmul_quantize_q8_amd as q
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    names = subprocess.run([nm, "-C", q.LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"void qmm::(k_experts_(?:few|matmul|matmul_k|stream)<.*>)(?=\(|$)", names, re.M))
    assert len(built) > 100 and built == {c[0] for c in CASES}
    norms = set(re.findall(r"void qmm::(k_rms_norm<.*>)(?=\(|$)", names, re.M))
    assert len(norms) == 24 and norms == {c[0] for c in NORMS}


def _ids(rng, T, top, E):
    """Experts of T * top / E rows, each a few more or fewer than its neighbours, so that their last tiles hold 1 to
    64 rows; every 50th pair has no expert."""
    pairs = T * top
    if pairs <= 64:
        ids = rng.integers(0, E, pairs)
    else:
        share = 1 + 0.02 * np.arange(E) + 0.3 * rng.random(E)
        counts = (pairs * share / share.sum()).astype(int)
        ids = np.concatenate([np.repeat(np.arange(E), counts), np.full(pairs - counts.sum(), E - 1)])
        ids[::50] = -1
    return rng.permutation(ids).reshape(T, top).astype(np.int32)


@functools.lru_cache(None)
def _pool(orc, fmt, K):
    """Three matrices of the most rows that a case of this format and K has, packed [3][rows][row bytes]."""
    rows = max(c[5] for c in CASES if c[1] == fmt and c[6] == K)
    values = np.random.default_rng(K).standard_normal((3 * rows, K)) * K ** -0.5
    return np.asarray(orc.quantize_w(fmt, values.astype(np.float32))).reshape(3, rows, -1)


def _some(ids, E):
    """Which pairs are compared: of each expert the first and the last 70 rows in the order of the pairs."""
    flat = ids.reshape(-1)
    pick = flat < 0
    for e in range(E):
        rows = np.flatnonzero(flat == e)
        pick[rows[:70]] = pick[rows[-70:]] = True
    return pick.reshape(ids.shape)


def _launched(torch, call):
    """Names of the kernels of a call."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.name for e in p.events() if e.device_type == torch.autograd.DeviceType.CUDA]


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,fmt,T,top,E,N,K,per_pair", CASES, ids=[f"{c[0]}-{c[2]}x{c[5]}x{c[6]}" for c in CASES])
def test_kernel(env, kernel, fmt, T, top, E, N, K, per_pair):
    torch, q, orc = env
    _say(kernel, fmt, T, top, E, N, K, per_pair)
    rng = np.random.default_rng(T + N + K)
    packed = [_pool(orc, fmt, K)[e % 3, :N] for e in range(E)]             # experts' matrices, the same for every third
    room = np.full((E, N + -N % 8, packed[0].shape[1]), 255, np.uint8)     # whole 16 bytes apart
    room[:, :N] = packed
    w = _dev(torch, room)[:, :N]
    act = q.ACT_FORMAT[fmt]
    xq = np.asarray(orc.quantize_x(fmt, rng.standard_normal((T * top if per_pair else T, K)).astype(np.float32)))
    xq = xq.reshape(-1, q.row_bytes(act, K))
    ids = _ids(rng, T, top, E)
    y, plan = torch.full((T, top, N), float("nan"), device="cuda"), q.experts_plan(T, top, E)
    x_d, ids_d = _dev(torch, xq), _dev(torch, ids)
    q.qmm_experts_plan(ids_d, E, plan)
    names = _launched(torch, lambda: q.EXPERTS_MATMUL[fmt](w, x_d, ids_d, plan, y))
    got = y.double().cpu().numpy()
    assert not np.isnan(got).any()
    pick = _some(ids, E)
    columns = np.unique(np.r_[:min(N, 40), max(0, N - 140):N, :N:7])       # the first and the last workgroup's, some between
    want, mag = ref.experts(orc, fmt, [np.ascontiguousarray(m[columns]) for m in packed], xq, np.where(pick, ids, -1),
                            columns.size, K, per_pair)
    # integer block sums are exact; two terms a block, each of three f32 steps, and the sum over the blocks
    bound = (2 * (K // q.BLOCK_VALUES[act]) + 8) * 2.0 ** -24 * mag + 2.0 ** -149
    off = np.abs(got[..., columns] - want)[pick] / bound[pick]
    assert np.all(off <= 1), float(off.max())
    assert np.all(got[ids < 0] == 0)
    # the name from the profiler, where it records this process
    assert not names or [n for n in names if kernel in n], names


@pytest.mark.gpu
@pytest.mark.parametrize("kernel,dtype,fmt,T,K", NORMS, ids=[f"{c[0]}-{c[3]}x{c[4]}" for c in NORMS])
def test_norm_kernel(env, kernel, dtype, fmt, T, K):
    torch, q, orc = env
    _say(kernel, dtype, fmt, T, K)
    rng = np.random.default_rng(T + K)
    x, xf = _rows(torch, rng, (T, K), dtype, pad=4)
    r, rf = _rows(torch, rng, (T, K), dtype, sigma=3.0)
    w = _dev(torch, (1 + 0.2 * rng.standard_normal(K)).astype(np.float32))
    xq = torch.full((T, q.row_bytes(fmt, K)), 255, dtype=torch.uint8, device="cuda")
    s, y = torch.empty_like(r), torch.empty_like(r)
    names = _launched(torch, lambda: q.RMS_NORM[fmt](x, w, xq, residual=r, sum=s, y=y, eps=1e-5))
    _norm_check(torch, q, orc, fmt, dtype, x, xf, r, rf, w, 1e-5, 0.0, s, y, xq)
    assert not names or [n for n in names if kernel in n], names
