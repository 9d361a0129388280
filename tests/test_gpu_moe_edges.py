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
