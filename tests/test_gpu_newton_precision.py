"""What the orthogonalised update keeps in more than fp16's 11 bits, seen in 32-bit
weights: from zeros, w <- 0 - lr scale O(g) with lr scale = -1 is O(g) before any rounding.

X's second word by itself: steps with b = c = 0 leave X as it was.  Two fp16 words are
off by 2^-23 of a number, one by 2^-12.  The polynomial's diagonal by itself: rows that
do not overlap and numbers that fp16 holds make X X^T diagonal and exact, and a cubic step
a s + b s^3.  Sums in 32 bits (a part of a matrix's squares, a thread's some 100 of them, and
ten roundings after) leave both below 2^-18 of themselves, where a word or the diagonal
in fp16 would leave 2^-12 / sqrt(3) = 1.4e-4.

The whole: the same roundings done by plain operations, in other orders of sums, are
off by as much (a quarter is allowed for chance, as some 64 directions of the smallest carry it); without
the 32-bit diagonal they are off by 1.8 times that (checked: 1.5)."""
import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_newton import CUBIC, QUINTIC, call, exact, gradient

pytestmark = pytest.mark.gpu

# small ones (whole on an SM) and larger ones, of either orientation, tiles with edges
SHAPES = [(2, 64, 64), (3, 128, 256), (2, 256, 128), (1, 104, 200), (2, 257, 512), (1, 129, 1000), (2, 300, 296), (1, 1000, 136), (1, 584, 584), (3, 520, 1416),
          (2, 1416, 520)]


def orthogonalised(g, steps):
    w, m = torch.zeros(g.shape, device="cuda"), torch.zeros(g.shape, device="cuda")
    ws = ep.alloc_orthogonalize_workspace(g.shape)
    ws.fill_(0xFF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_muon_update(g, m, w, None, steps, ws, lr=1.0, scale=-1.0, momentum=0.0, nesterov=False, status=status)
    assert ep.ep_read_status(status) == ep.EP_OK
    return w.double()


def rel(a, b):
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_words_of_x(shape, dtype):
    g = gradient(sum(shape), *shape, dtype=dtype)
    for steps in ([(1.0, 0.0, 0.0)] * 3, [(0.75, 0.0, 0.0), (1.25, 0.0, 0.0)]):
        assert rel(orthogonalised(g, steps), exact(g, steps)) < 2.0 ** -18


@pytest.mark.parametrize("shape", SHAPES)
def test_diagonal(shape):
    count, M, N = shape
    S = min(M, N)
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    # sizes of 8 bits within a factor of 8; element (i, i + shift) of the matrix whose rows are the smaller side
    sizes = torch.randint(32, 256, (count, S), generator=gen, device="cuda").float() * 2.0 ** -12
    x = torch.zeros((count, S, max(M, N)), device="cuda")
    at = torch.randperm(max(M, N), generator=gen, device="cuda")[:S]
    x[:, torch.arange(S, device="cuda"), at] = sizes
    g = (x.transpose(1, 2) if M > N else x).contiguous().bfloat16()
    # (singular values of about S^-1/2: the cubic term has to show)
    steps = [(1.5, -0.5 * S, 0.0)]
    assert rel(orthogonalised(g, steps), exact(g, steps)) < 2.0 ** -18


def emulated(g, steps, low=True, diagonal=True):
    """The design's roundings: fp16 operands 2^8 times as large, X in two words, P's diagonal in 32 bits."""
    held, half = 256.0, lambda v: v.half().double()  # noqa: E731
    tall = g.shape[-2] > g.shape[-1]
    x = (g.transpose(-1, -2) if tall else g).double()
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + 1e-7) * held
    for a, b, c in steps:
        hi = half(x)
        A = half(hi @ hi.transpose(-1, -2) / held)
        P = b * A + c * (A @ A) / held
        d = P.diagonal(dim1=-2, dim2=-1) / held if diagonal else torch.zeros_like(P[..., 0])
        if diagonal:
            P = P - torch.diag_embed(P.diagonal(dim1=-2, dim2=-1))
        x = (a + d).unsqueeze(-1) * (hi + half(x - hi) if low else hi) + half(P) @ hi / held
    x = x / held
    return x.transpose(-1, -2) if tall else x


@pytest.mark.parametrize("shape", SHAPES)
def test_quintic_is_off_by_the_designs_roundings(shape):
    g = gradient(1 + sum(shape), *shape, dtype=torch.float32)
    steps = [QUINTIC] * 5
    want = exact(g, steps)
    design = rel(emulated(g, steps), want)
    assert rel(emulated(g, steps, diagonal=False), want) > 1.5 * design
    assert rel(orthogonalised(g, steps), want) < 1.25 * design


def of_few_left(tiles, pairs):
    """Matrices of `tiles` tiles each that fill the pairs of SMs and leave a few."""
    return -(-pairs // tiles)


@pytest.mark.parametrize("M,N,tiles", [(520, 520, 6), (1000, 520, 6), (520, 776, 6), (264, 1416, 3), (1416, 264, 3)])
def test_a_last_wave_of_halves(M, N, tiles):
    """Stacks whose symmetric products leave a few tiles over a wave, which are cut in two: on and above the diagonal.  As
    alone, where tiles are narrow."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    count = of_few_left(tiles, pairs)
    assert 0 < 2 * (count * tiles % pairs) <= pairs
    g = gradient(M + N, count, M, N)
    for steps in ([QUINTIC] * 3, [CUBIC] * 2):
        out = call(g, steps)
        for z in range(count):
            if z < 2 or z > count - 4:
                assert torch.equal(call(g[z:z + 1].contiguous(), steps)[0], out[z]), z
        want = exact(g, steps)
        assert rel(out.double(), want) < 0.0025   # bf16's 2^-8 / sqrt(3) = 0.00226, and 0.001 beside it


@pytest.mark.parametrize("M,N", [(40, 264), (264, 40), (129, 136)])
def test_many_matrices_of_one_tile(M, N):
    g = gradient(M, 700, M, N)
    out = call(g, [QUINTIC] * 4)
    for z in (0, 350, 690, 699):
        assert torch.equal(call(g[z:z + 1].contiguous(), [QUINTIC] * 4)[0], out[z])
