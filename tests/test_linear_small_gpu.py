"""Projections of few rows or features: operands of less than 128 KB, at the end of the
memory that is mapped, before values that are not theirs, among other allocations."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MAPPED = 16 << 20     # an allocation of its own


@pytest.fixture(scope="module")
def ssd():
    import selective_state_space_05_gb300 as m
    return m


def at_the_end(t):
    """A copy of t whose last element is the last of its allocation."""
    buf = torch.empty(MAPPED // t.element_size(), dtype=t.dtype, device="cuda")
    got = buf[buf.numel() - t.numel():].view(t.shape)
    got.copy_(t)
    return got


def close(got, a, b, what):
    """got against a b^T in 64 bits: a sum of K products in fp32 (2^-23 of the sum of
    their sizes a product at most, six products and three planes for fp32), rounded
    once."""
    a, b = a.double(), b.double()
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = torch.finfo(got.dtype).eps / 2 * ref.abs() + (a.shape[1] + 8) * 2.0 ** -23 * size
    off = (got.double() - ref).abs()
    assert (off <= bound).all(), f"{what}: {float((off / bound).max()):.3g} times its bound"


def check(ssd, x, w, dout):
    close(ssd.linear_fwd(x, w), x, w, "out")
    g = ssd.linear_bwd(dout, x, w)
    close(g["dx"], dout, w.t(), "dx")
    close(g["dweight"], dout.t(), x.t(), "dweight")


def operands(M, K, N, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*s, generator=gen, device="cuda").to(dtype)
            for s in ((M, K), (N, K), (M, N))]


SIZES = [(9, 5120, 64), (17, 2560, 352), (33, 128, 648), (120, 512, 8), (127, 256, 1000),
         (128, 128, 128), (210, 128, 648), (210, 256, 128), (300, 64, 40)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_at_the_end_of_memory(ssd, dtype, M, K, N):
    x, w, dout = (at_the_end(t) for t in operands(M, K, N, dtype, M + K))
    check(ssd, x, w, dout)


@pytest.mark.parametrize("M,K,N", SIZES)
def test_what_lies_behind_stays_out(ssd, M, K, N):
    """Rows of NaN behind each operand."""
    got = []
    for t in operands(M, K, N, BF, M):
        buf = torch.full((t.shape[0] + 140, t.shape[1]), float("nan"), dtype=BF, device="cuda")
        buf[:t.shape[0]] = t
        got.append(buf[:t.shape[0]])
    check(ssd, *got)


def test_among_other_allocations(ssd):
    """Holes between what is mapped, other ones each time."""
    gen = torch.Generator().manual_seed(1)
    for rep in range(12):
        torch.cuda.empty_cache()
        sizes = torch.randint(1, 3 << 20, (40,), generator=gen).tolist()
        other = [torch.full((n,), float("nan"), device="cuda") for n in sizes]
        hold = other[::5]
        del other
        torch.cuda.empty_cache()
        for M, K, N in SIZES:
            check(ssd, *operands(M, K, N, BF, rep))
        del hold
