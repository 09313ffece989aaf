"""softplus of the step as every kernel computes it, against 64 bits.  With A = 0, x = B = 1 and no state
before, one step's state is softplus(delta + delta_bias) itself; delta is 0 and delta_bias the value.

The bound is step_dt's of serving_ref.py, (8 + 3 |v|) roundings of 2^-24 relative to the result, and two more for
the products with x and B."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DIM = 16384


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_61_amd as ssm
    ssm.load_library()


@pytest.fixture(scope="module")
def ssm():
    import selective_state_space_61_amd as m
    return m


def values():
    """Ordinary steps, all of -20..25, and where 1 + e^v passes a power of two or leaves fp32's whole numbers."""
    rng = np.random.default_rng(3)
    v = [rng.uniform(-20.0, 25.0, 4096), rng.uniform(-8.0, 0.0, 2048), rng.uniform(16.5, 17.5, 2048)]
    v += [np.log(2.0 ** k - rng.uniform(0.0, 1.0, 256)) for k in range(2, 26)]
    v = np.concatenate(v)
    return torch.from_numpy(np.concatenate([v, rng.uniform(-2.0, 3.0, DIM - v.size)]).astype(np.float32))


def check(got, v, what, steps=0.0):
    """got: the values computed for v, `steps` more relative roundings of its type allowed."""
    ref = torch.logaddexp(v.double(), torch.zeros(v.shape, dtype=torch.float64))
    tol = (ref * ((10 + 3 * v.double().abs()) * R.U + steps))
    ratio = (R.f64(got).reshape(v.shape) - ref).abs() / tol
    print(f"  {what}: worst error {ratio.max().item():.3f} of its bound, at {v[ratio.argmax()].item()!r}", flush=True)
    assert (ratio <= 1.0).all()


def one(*shape, dtype):
    return torch.ones(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype,layout", [("f32", "auto"), ("f32", "time_scan"), ("bf16", "channel_lanes"),
                                          ("bf16", "state_rows")])
def test_scan(ssm, dtype, layout):
    v, t = values(), DT[dtype]
    x, b = one(1, 1, DIM, dtype=t), one(1, 1, 16, dtype=t)
    _, h = ssm.ssm_scan_fwd(x, 0 * x, torch.zeros(DIM, 16, device="cuda"), b, b, delta_bias=v.cuda(), delta_softplus=True,
                            layout=layout)
    check(h[0, :, 0], v, f"scan {dtype} {layout}")
    assert (h == h[:, :, :1]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 16, 64])
def test_scan_packed(ssm, n, dtype):
    v, t = values(), DT[dtype]
    x, b, h = one(1, DIM, dtype=t), one(1, n, dtype=t), torch.zeros(1, DIM, n, device="cuda")
    ssm.ssm_scan_packed_fwd(x, 0 * x, torch.zeros(DIM, n, device="cuda"), b, b, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                            delta_bias=v.cuda(), delta_softplus=True, cache=h)
    check(h[0, :, n - 1], v, f"packed scan {dtype} dstate {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cached", [False, True])
def test_scan_step(ssm, cached, dtype):
    v, t = values(), DT[dtype]
    x, b, h, a = one(1, DIM, dtype=t), one(1, 16, dtype=t), torch.zeros(1, DIM, 16, device="cuda"), torch.zeros(DIM, 16, device="cuda")
    if cached:
        ssm.ssm_state_update_cache(h, None, x, 0 * x, a, b, b, delta_bias=v.cuda(), delta_softplus=True)
    else:
        ssm.ssm_state_update(h, x, 0 * x, a, b, b, delta_bias=v.cuda(), delta_softplus=True)
    check(h[0, :, 0], v, f"step {dtype}, cache {cached}")


@pytest.mark.parametrize("cached", [False, True])
def test_ssd_step(ssm, cached):
    v = values()
    x, b = one(1, DIM, 16, dtype=torch.bfloat16), one(1, 1, 64, dtype=torch.bfloat16)
    dt, a, h = torch.zeros(1, DIM, dtype=torch.bfloat16, device="cuda"), torch.zeros(DIM, device="cuda"), torch.zeros(1, DIM, 16, 64, device="cuda")
    if cached:
        ssm.ssm_ssd_state_update_cache(h, None, x, dt, a, b, b, dt_bias=v.cuda(), dt_softplus=True)
    else:
        ssm.ssm_ssd_state_update(h, x, dt, a, b, b, dt_bias=v.cuda(), dt_softplus=True)
    check(h[0, :, 0, 0], v, f"SSD step, cache {cached}")


def test_ssd_layer(ssm):
    # the chunk's products take bf16 operands: dt x is rounded once to bf16
    v = values()
    x, b = one(1, 1, DIM, 16, dtype=torch.bfloat16), one(1, 1, 1, 32, dtype=torch.bfloat16)
    _, h = ssm.ssm_ssd_fwd(x, torch.zeros(1, 1, DIM, dtype=torch.bfloat16, device="cuda"), torch.zeros(DIM, device="cuda"), b, b,
                           dt_bias=v.cuda(), dt_softplus=True)
    check(h[0, :, 0, 0], v, "SSD layer", 1.01 * R.half_step(torch.bfloat16))


@pytest.mark.parametrize("dtype,layout", [("f32", "channel_lanes"), ("bf16", "channel_lanes"), ("bf16", "state_rows")])
def test_scan_backward(ssm, dtype, layout):
    # y = dt sum_n B_n C_n x, with sum_n B_n C_n = 1: dx = dt dy, rounded once to x's type
    v, t = values(), DT[dtype]
    x, b = one(1, 1, DIM, dtype=t), one(1, 1, 16, dtype=t)
    g = ssm.ssm_scan_bwd(x, 0 * x, torch.zeros(DIM, 16, device="cuda"), b, b / 16, x, delta_bias=v.cuda(), delta_softplus=True,
                         layout=layout)
    # (16 equal terms of dt / 16: their sums are 15 roundings more)
    check(g["dx"][0, 0], v, f"backward {dtype} {layout}", 16 * R.U + (1.01 * R.half_step(t) if dtype == "bf16" else 0.0))
