"""Long sums of the projections: the tensor core's fp32 sum rounds towards
zero at every step, which sums of one sign show.  An accumulator takes 64 MMAs
(of 16 products each; fp32 operands 32) where the result is kept in fp32 and 1024
where it is rounded to bf16; the accumulators' totals are added to nearest."""
import pytest
import torch

import block_testutil as bt

pytestmark = pytest.mark.gpu

F32, BF = torch.float32, torch.bfloat16


def ones_like_values(*shape, seed, dt):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda").uniform_(0.7, 1.3, generator=g).to(dt)


@pytest.mark.parametrize("dt", [F32, BF])
def test_results_kept_in_fp32(dt):
    """76 tiles of 256 x 256, no split of K: 1024 MMAs a product of planes.  A
    run's partial sum after i of 64 MMAs is i / 64 of the run's, each truncated by
    up to 2^-23 of it: 32 of 2^-23, 64 of 2^-24 in all; then a rounding a run,
    and of the fp32 operands' six products the small ones' own (2^-8 of it).
    Without runs the sum is short by 1024 * 2^-24 at most, 200 * 2^-24 or so."""
    import selective_state_space_05_gb300 as ssd
    M, K, N = 4864, 16384, 1024
    x, w = ones_like_values(M, K, seed=1, dt=dt), ones_like_values(N, K, seed=2, dt=dt)
    res = torch.zeros(M, N, device="cuda")
    out = ssd.linear_fwd(x, w, residual=res)
    ssd.scan_status()
    ref = (x.double() @ w.double().t()).cpu()
    bt.assert_within(out, ref, ref.abs(), 64 + K // 1024 + 4, "out")


@pytest.mark.parametrize("tokens", [2 ** 17 + 5, 2 ** 24])
def test_weight_gradient_of_many_tokens(tokens):
    """bf16 dW sums over the tokens.  Each accumulator is short by at most
    1024 / 2 * 2^-23 of its sum, 2^-14 (a 32nd of bf16's least half step);
    the rest is the result's one rounding."""
    import selective_state_space_05_gb300 as ssd
    x = ones_like_values(tokens, 64, seed=3, dt=BF)
    do = ones_like_values(tokens, 64, seed=4, dt=BF)
    got = ssd.linear_bwd(do, x, None, need_dx=False)["dweight"]
    ssd.scan_status()
    ref = torch.zeros(64, 64, dtype=torch.float64, device="cuda")
    for a, b in zip(do.split(1 << 20), x.split(1 << 20)):
        ref += a.double().t() @ b.double()
    ref = ref.cpu()
    bt.assert_within(got, ref, ref.abs(), 0, "dweight", extra=2.0 ** -14 * ref.abs())


def test_forward_of_many_features():
    import selective_state_space_05_gb300 as ssd
    K = 2 ** 24
    x, w = ones_like_values(70, K, seed=5, dt=BF), ones_like_values(40, K, seed=6, dt=BF)
    out = ssd.linear_fwd(x, w)
    ssd.scan_status()
    ref = torch.zeros(70, 40, dtype=torch.float64, device="cuda")
    for a, b in zip(x.split(1 << 19, 1), w.split(1 << 19, 1)):
        ref += a.double() @ b.double().t()
    ref = ref.cpu()
    bt.assert_within(out, ref, ref.abs(), 0, "out", extra=2.0 ** -14 * ref.abs())


@pytest.mark.parametrize("K", [512, 2048, 5120, 10576])
@pytest.mark.parametrize("dt,units", [(F32, 10), (BF, 20)])
def test_results_kept_in_fp32_of_both_signs(dt, units, K):
    """The relative error of the whole result that the kernel's comment states:
    4.8e-7 (8 * 2^-24) for fp32 operands, 1.0e-6 (17 * 2^-24) for bf16 ones; the
    bounds fail with sums twice as long."""
    import selective_state_space_05_gb300 as ssd
    g = torch.Generator("cuda").manual_seed(K)
    x = torch.randn(900, K, generator=g, device="cuda").to(dt)
    w = (torch.randn(1000, K, generator=g, device="cuda") * K ** -0.5).to(dt)
    ref = x.double() @ w.double().t()
    out = ssd.linear_fwd(x, w, residual=torch.zeros(900, 1000, device="cuda"))
    ssd.scan_status()
    assert float((out.double() - ref).norm() / ref.norm()) <= units * bt.U32


def test_equal_bits_on_every_call():
    """The sums' order is fixed, whatever else the GPU does."""
    import selective_state_space_05_gb300 as ssd
    for dt, M, K, N, act in ((BF, 8192, 2560, 2560, None), (F32, 1023, 512, 1096, "silu"),
                             (BF, 1021, 5120, 2560, "gelu")):
        x, w = torch.randn(M, K, device="cuda").to(dt), torch.randn(N, K, device="cuda").to(dt)
        do = torch.randn(M, N, device="cuda").to(dt)

        def step():
            out, pre = ssd.linear_fwd(x, w, activation=act, save_pre=True)
            g = ssd.linear_bwd(do, x, w, activation=act, pre=pre, need_dbias=True)
            return [out, pre, g["dx"], g["dweight"], g["dbias"]]

        want = step()
        for _ in range(10):
            torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(7)   # out of the L2
            assert all(torch.equal(a, b) for a, b in zip(step(), want))
