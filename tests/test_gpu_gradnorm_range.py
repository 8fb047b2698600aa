"""Gradients' norms and clipping at the ends of fp32's range: norms beyond it, zeros of
both signs, values whose squares are far below it.  Bounds as in test_gpu_gradnorm.py;
a sum of scaled squares is exact to the same 33 U."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from objective_ref import U  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def norm64(ts):
    return float(np.sqrt(sum(float(t.double().square().sum()) for t in ts)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_norm_beyond_32_bits_is_reported_and_not_applied(dtype):
    # two finite elements whose norm is 4.2e38: what the caller sees is inf
    big = torch.zeros(1000, dtype=DT[dtype], device="cuda")
    big[3], big[700], big[999] = 3e38, -3e38, 1.5
    other = torch.full((1000,), 2.0, dtype=DT[dtype], device="cuda")
    kept = big.clone()
    out = [torch.empty(1000, device="cuda") for _ in range(2)]
    norms = pkg.clip_grads([[big], [other]], 1.0, out=[[out[0]], [out[1]]])
    assert float(norms[0]) == np.inf and float(norms[1]) == pytest.approx(np.sqrt(4000.0), rel=20 * U)
    assert torch.equal(out[0], kept.float())
    assert float(out[1].norm()) == pytest.approx(1.0, rel=1e-5)
    norms = pkg.clip_grads([[big], [other]], 1.0)
    assert float(norms[0]) == np.inf and torch.equal(big, kept)
    assert float(pkg.grad_norm([kept])) == np.inf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_norm_just_within_32_bits_is_applied(dtype):
    t = torch.zeros(1000, dtype=DT[dtype], device="cuda")
    t[3], t[700] = 2.375e38, -2.375e38  # norm 3.36e38, largest float 3.40e38
    want = norm64([t])
    out = torch.empty(1000, device="cuda")
    got = float(pkg.clip_grads([t], 1e30, out=[out]))
    assert abs(got - want) <= 18 * U * want
    ref = t.double() * (float(np.float32(1e30)) / want)
    assert ((out.double() - ref).abs() <= 20 * U * ref.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_zeros_of_both_signs(dtype):
    z = torch.zeros(100003, dtype=DT[dtype], device="cuda")
    m = -z
    assert torch.signbit(m).all()
    assert pkg.grad_norm([[z], [m], [z, m]]).tolist() == [0.0, 0.0, 0.0]
    m[77] = -0.5
    assert float(pkg.grad_norm([m])) == 0.5
    m[77] = -0.0
    pkg.clip_grads([m], 1.0)
    assert torch.signbit(m).all() and m.eq(0).all()


SMALL = {"bf16": [1e-12, 1e-25, 2.0 ** -126, 2.0 ** -133], "f16": [2.0 ** -24, 2.0 ** -14],
         "f32": [1e-12, 1e-25, 2.0 ** -126, 2.0 ** -149]}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_small_values(dtype):
    gen = torch.Generator(device="cuda").manual_seed(0)
    for size in SMALL[dtype]:
        for n in (1, 9, 1000, 70001):
            t = (torch.randn(n, generator=gen, device="cuda").double() * size).to(DT[dtype])
            want = norm64([t])
            got = float(pkg.grad_norm([t]))
            assert abs(got - want) <= 18 * U * want + 2.0 ** -149, (size, n, got, want)
            # beside one element that is not small
            t[n // 2] = 1.0
            assert abs(float(pkg.grad_norm([t])) - norm64([t])) <= 18 * U * norm64([t])


def test_small_and_large_batches_side_by_side():
    # a thread's elements are 2^-149 to 2^120 apart
    t = torch.zeros(1 << 20, device="cuda")
    t[::2] = 2.0 ** -149
    t[5::4099] = 2.0 ** 62
    t[7::70001] = -(2.0 ** 120)
    want = norm64([t])
    assert abs(float(pkg.grad_norm([t])) - want) <= 18 * U * want
