"""Calls of the mixture-of-experts operators at the ends of what their contracts allow, on an MI355X."""
import numpy as np
import pytest

import moe_ref as ref
from test_gpu_moe import _counted, _dev, _say, env          # noqa: F401  (env: the fixture)

pytestmark = pytest.mark.gpu


# Gates for which e^-g, or the erfc of the GELU, leaves the normal f32 values while the activation does not (first
# half), and where the activation itself is below them (second half), with factors that bring the products back.
TAILS = {"silu": ((-92.0, -88.8, 1e37), (-103.0, -95.0, 3e38)),
         "gelu": ((-13.3, -13.05, 1e38), (-14.2, -13.95, 3e38)),
         "gelu_tanh": ((-10.2, -10.06, 1e37), (-10.6, -10.35, 3e38))}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["q8_0", "q8_k"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_glu_far_gates(env, act, fmt, dtype):
    """The relative error r of a value is that of the whole range: 16 f32 steps times the 104 that a far gate's
    exponent, rounded to 2^-24 of itself, can amplify one by; the blocks then as at any other gate."""
    torch, q, _ = env
    _say("glu far", act, fmt, dtype)
    V = ref.VALUES[fmt]
    g, u = np.empty((2, V), np.float32), np.empty((2, V), np.float32)
    for i, (lo, hi, factor) in enumerate(TAILS[act]):
        g[i], u[i] = np.linspace(lo, hi, V), factor * np.where(np.arange(V) % 3, 1, -1)
    gate, up = _dev(torch, g, dtype), _dev(torch, u, dtype)
    xq = torch.zeros(2, q.row_bytes(fmt, V), dtype=torch.uint8, device="cuda")
    q.GLU[fmt](gate, up, xq, act=act)
    want = ref.activation(gate.float().cpu().numpy(), act) * up.double().cpu().numpy()
    values, d = ref.decoded(xq.cpu().numpy(), fmt)
    r = 16 * 104 * 2.0 ** -24
    amax = np.abs(want).max(1)
    assert np.all(amax > 1e-5)
    step, tiny = (2.0 ** -11, 2.0 ** -25) if fmt == "q8_0" else (2.0 ** -23, 0)
    assert np.all(np.abs(d[:, 0] - amax / 127) <= (step + 2 * r) * amax / 127 + tiny)
    assert np.all(np.abs(values - want) <= (amax / 127 * (0.5 + 127 * (step + 2 * r)) + 127 * tiny)[:, None])


def test_one_plan_buffer_for_every_batch(env):
    """A buffer made for the largest batch, used by smaller ones in turn: exact products of whole numbers."""
    torch, q, _ = env
    top, E, most = 4, 64, (1 << 16) + 1
    plan = q.experts_plan(most, top, E)
    for T in (most, most - 1, 3, 700, 20, 16384):
        _say("plan buffer", T)
        ids = np.random.default_rng(T).integers(-1, E, (T, top)).astype(np.int32)
        w, x, sums = _counted(torch, q, T, top, E)
        y = torch.full((T, top, 8), float("nan"), device="cuda")
        ids_d = _dev(torch, ids)
        q.qmm_experts_plan(ids_d, E, plan)
        q.qmm_experts_matmul_q8_0(w, x, ids_d, plan, y)
        want = ((ids + 1) * sums[:, None]).astype(np.float32)              # -1: zero
        assert np.array_equal(y.cpu().numpy(), np.repeat(want[..., None], 8, 2))


@pytest.mark.parametrize("N", [7, 8])
def test_combine_of_one_row_of_any_stride(env, N):
    """A row's stride that no size could hold is not read."""
    torch, q, _ = env
    _say("combine one row", N)
    y, w, r = torch.randn(1, 3, N, device="cuda"), torch.rand(1, 3, device="cuda"), torch.randn(1, N, device="cuda")
    out, far = torch.empty(1, N, device="cuda"), torch.empty(N, device="cuda").as_strided((1, N), (1 << 60, 1))
    q.qmm_experts_combine(y, w, out, residual=r)
    q.qmm_experts_combine(y, w, far, residual=r.as_strided((1, N), (1 << 60, 1)))
    assert torch.equal(out, far) and torch.isfinite(out).all()


@pytest.mark.parametrize("T", [1, 40])
def test_experts_of_one_matrix_of_any_stride(env, T):
    """One expert's matrix, a view of rows of matrices that lie at no whole 16 bytes."""
    torch, q, _ = env
    _say("one matrix", T)
    w, x, sums = _counted(torch, q, T, 1, 3, N=9, K=64)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    plan = q.experts_plan(T, 1, 1)
    q.qmm_experts_plan(ids, 1, plan)
    for one in (w[:1, :7], w[0, :7].as_strided((1, 7, 68), (1 << 60, 68, 1))):
        assert one.stride(0) % 16 != 0 or one.stride(0) == 1 << 60
        y = torch.full((T, 1, 7), float("nan"), device="cuda")
        q.qmm_experts_matmul_q8_0(one, x, ids, plan, y)
        assert np.array_equal(y.cpu().numpy()[:, 0], np.repeat(sums[:, None], 7, 1).astype(np.float32))


def _ones(torch, fmt, E, N, blocks):
    """Matrices of codes that stand for 1, expert e's scale 2^(e % 3): [E][N][row bytes]."""
    scale = {e: [int(b) for b in np.float16(2.0 ** e).reshape(1).view(np.uint8)] for e in range(3)}
    block = {"q8_0": lambda d: d + [1] * 32, "q4_0": lambda d: d + [0x99] * 16,
             "q4_k": lambda d: d + [0, 0] + [1] * 4 + [0] * 4 + [1] * 4 + [0x11] * 128,          # scales 1, minima 0
             "q6_k": lambda d: [0x11] * 128 + [0xaa] * 64 + [1] * 16 + d}[fmt]                   # 33 - 32
    three = torch.tensor([block(scale[e]) for e in range(3)], dtype=torch.uint8, device="cuda")
    row = three.repeat(1, blocks)[torch.arange(E, device="cuda") % 3]
    return row[:, None].expand(E, N, row.shape[1]).contiguous()


def _signs(torch, fmt, T, blocks):
    """Rows of -1, 0 and 1 with scale 1, and their sums."""
    values = 256 if fmt.endswith("_k") else 32
    codes = torch.randint(-1, 2, (T, blocks, values), dtype=torch.int8, device="cuda")
    if values == 32:
        x = torch.empty(T, blocks, 34, dtype=torch.uint8, device="cuda")
        x[..., 0], x[..., 1] = 0, 0x3c
        x[..., 2:] = codes.view(torch.uint8)
    else:
        x = torch.empty(T, blocks, 292, dtype=torch.uint8, device="cuda")
        x[..., :4] = torch.tensor([0, 0, 0x80, 0x3f], dtype=torch.uint8, device="cuda")
        x[..., 4:260] = codes.view(torch.uint8)
        x[..., 260:] = codes.view(T, blocks, 16, 16).sum(-1, dtype=torch.int16).view(torch.uint8).view(T, blocks, 32)
    return x.view(T, -1), codes.sum((1, 2), dtype=torch.int64)


@pytest.mark.parametrize("fmt,T,E,N,blocks", [
    ("q8_0", 3855, 240, 8, 32768), ("q4_0", 3855, 240, 8, 32767), ("q8_0", 3855, 100, 8, 32768),     # tiles of 16, of 32
    ("q8_0", 3854, 20, 8, 32774), ("q4_0", 4200, 1, 520, 30070),                          # the prefill tiles of 32 and 128
    ("q6_k", 3855, 240, 8, 3815), ("q4_k", 4200, 1, 700, 3501), ("q6_k", 4200, 1, 700, 3501)])       # of 16, 64, 128
def test_experts_of_nearly_4_gib_of_rows(env, fmt, T, E, N, blocks):
    """Rows whose offsets pass 2^31 and end just below 2^32 bytes: exact products of whole numbers."""
    torch, q, _ = env
    _say("4 GiB", fmt, T, E, N, blocks)
    w = _ones(torch, fmt, E, N, blocks)
    x, sums = _signs(torch, fmt, T, blocks)
    assert 0.99 * 2 ** 32 < x.numel() < 2 ** 32
    ids = torch.randint(0, E, (T, 1), dtype=torch.int32, device="cuda")
    plan, y = q.experts_plan(T, 1, E), torch.full((T, 1, N), float("nan"), device="cuda")
    q.qmm_experts_plan(ids, E, plan)
    q.EXPERTS_MATMUL[fmt](w, x, ids, plan, y)
    want = (sums * 2 ** (ids[:, 0] % 3)).float()
    assert torch.equal(y[:, 0], want[:, None].expand(T, N))


def test_norm_of_more_rows_than_a_grid(env):
    """Workgroups that take a second row, against the same rows in calls of fewer."""
    torch, q, _ = env
    T, K = (1 << 20) + 77, 64
    _say("norm of many rows", T)
    x, r = torch.randn(T, K, device="cuda"), torch.randn(T, K, device="cuda")
    xq, s, y = torch.zeros(T, 68, dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    q.qmm_rms_norm_q8_0(x, None, xq, residual=r, sum=s, y=y)
    for part in (slice(0, 1000), slice((1 << 20) - 500, T)):
        n = len(range(*part.indices(T)))
        xq2, s2, y2 = torch.empty(n, 68, dtype=torch.uint8, device="cuda"), x.new_empty(n, K), x.new_empty(n, K)
        q.qmm_rms_norm_q8_0(x[part], None, xq2, residual=r[part], sum=s2, y=y2)
        assert torch.equal(xq[part], xq2) and torch.equal(s[part], s2) and torch.equal(y[part], y2)
    want = ref.norm((x[-77:] + r[-77:]).cpu().numpy(), None, 1e-6)
    assert np.all(np.abs(y[-77:].cpu().numpy() - want) <= (2.0 ** -24 + 1e-12) * np.abs(want) + 2.0 ** -149)
