"""Schedules of Newton-Schulz coefficients other than the usual five steps, against the definition
in 64 bits.

X is read from fp32 weights that start at 0 and take a step of rate -1 with a momentum of 0, so
that no rounding of a result comes on top.  Errors are in X's norm.
  What the header promises for the roundings of the products: PROMISE below.
  `floor`: 22 bits of u and of what the products sum in fp32 leave a part nu of u's norm that is not
u's.  It grows like the singular values of its directions, by at most the product G of the slopes at
0, and until those reach order one: by 1 / the smallest of u's, times 8 for the steps from
there on, where a slope may still exceed 1.  nu = 2^-20: pairs of fp16 are off by 2^-23 of an element, the sums
of 24 products of 16 terms in Q X by 2^-23 of the running sum each time, 5 of those in the mean (their
root): 6 2^-23.  Where nu grows to order one X is as large as its directions are many."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding, muon  # noqa: E402

USUAL = (3.4445, -4.7750, 2.0315)
PROMISE = 2e-3  # of up to 128 rows or columns
PROMISE_MANY = 6e-3  # of more
PROMISE_EQUAL = 1.2e-2  # where most singular values are equal, or slopes pass 4


def exact(u, coefficients, eps=1e-7):
    """The definition: u [R, C] in 64 bits."""
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    for a, b, c in coefficients:
        if x.shape[0] <= x.shape[1]:
            g = x @ x.mT
            x = a * x + (b * g + c * (g @ g)) @ x
        else:
            g = x.mT @ x
            x = a * x + x @ (b * g + c * (g @ g))
    return x


def with_values(r, c, values, seed=0):
    """A matrix of these singular values."""
    g = torch.Generator().manual_seed(seed)
    m = min(r, c)
    left, _ = torch.linalg.qr(torch.randn(r, m, generator=g, dtype=torch.float64))
    right, _ = torch.linalg.qr(torch.randn(c, m, generator=g, dtype=torch.float64))
    return ((left * torch.as_tensor(values, dtype=torch.float64)) @ right.mT).float()


def x_of(u, coefficients):
    """X in 32 bits, as the step takes it off weights of 0."""
    w, m = torch.zeros_like(u), torch.zeros_like(u)
    factor = math.sqrt(max(1.0, u.shape[0] / u.shape[1]))
    plan = flce.muon_plan([w], [m], lr=-1.0 / factor, momentum=0.0, nesterov=False, steps=len(coefficients),
                          coefficients=list(coefficients))
    flce.muon_step(plan, [u], check=True)
    return w


def off(u, coefficients):
    """The error of X, and what the floor adds to the promise, both of X's norm."""
    near = exact(u, coefficients)
    norm = near.norm().item()
    least = (torch.linalg.svdvals(u.double())[-1] / u.double().norm()).item()
    grown = min(math.prod(max(1.0, abs(a)) for a, _, _ in coefficients), 8.0 / max(least, 1e-300))
    floor = min(2.0 ** -20 * grown, 2.0 * min(u.shape) ** 0.5) / norm
    return ((x_of(u, coefficients).double() - near).norm() / norm).item(), floor


#: four usual steps, then four whose product is largest for a singular value of 0.0141275, between
#: the points of a grid of 256: 52 times X there, 1.05 at its neighbours
PEAK = [USUAL] * 4 + [(0.3691, -0.2635, -0.4207), (0.2906, -1.0417, -0.2021), (0.2066, -0.809, 0.1765),
                      (0.2686, -1.4555, -0.7431)]


@pytest.mark.gpu
@pytest.mark.parametrize("r,c", [(64, 96), (96, 64), (16, 16)])
def test_products_of_the_steps_that_peak_anywhere(r, c):
    m, s = min(r, c), 0.0141275
    u = with_values(r, c, [math.sqrt(1 - (m - 1) * s * s)] + [s] * (m - 1)).cuda()
    error, floor = off(u, PEAK)
    assert error <= PROMISE + floor


def matrix(r, c, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    noise = torch.randn(r, c, generator=g)

    def directions(k):
        return torch.randn(r, k, generator=g) @ torch.randn(k, c, generator=g)
    return {"noise": lambda: noise, "same": lambda: torch.eye(r, c),
            "strong": lambda: directions(8) + 0.05 * noise,   # eight directions over noise
            "rank8": lambda: directions(8) + 0.003 * noise,   # over a thousandth of it
            "rank1": lambda: directions(1),                   # over nothing at all
            "decay": lambda: with_values(r, c, torch.logspace(0, -5, min(r, c)), seed)}[kind]()


SCHEDULES = {"usual 6": [USUAL] * 6, "usual 8": [USUAL] * 8, "usual 10": [USUAL] * 10, "usual 16": [USUAL] * 16,
             "cubic 16": [(1.5, -0.5, 0.0)] * 16, "quintic 16": [(1.875, -1.25, 0.375)] * 16,
             "mixed": [USUAL] * 7 + [(1.875, -1.25, 0.375)] * 3}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["noise", "strong", "rank8", "rank1", "decay"])
@pytest.mark.parametrize("r,c", [(64, 200), (128, 128), (300, 100), (128, 1544)])
@pytest.mark.parametrize("schedule", SCHEDULES)
def test_few_rows_and_many_steps(r, c, kind, schedule):
    error, floor = off(matrix(r, c, kind).cuda(), SCHEDULES[schedule])
    assert error <= PROMISE + floor


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [6, 11, 16])
def test_few_rows_beside_many_of_them(steps):
    """One call's matrices read X a few times or at every step: the same bits as each alone."""
    xs = [matrix(r, c, "strong", r).cuda() for r, c in ((300, 200), (40, 60), (128, 640), (200, 300), (7, 5))]
    got = flce.orthogonalize(xs, steps=steps, check=True)
    for x, y in zip(xs, got):
        assert torch.equal(y, flce.orthogonalize(x, steps=steps))

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["noise", "strong", "same", "rank8", "rank1", "decay"])
@pytest.mark.parametrize("r,c", [(300, 777), (640, 400), (129, 129)])
@pytest.mark.parametrize("schedule", SCHEDULES)
def test_many_rows_and_many_steps(r, c, kind, schedule):
    error, floor = off(matrix(r, c, kind).cuda(), SCHEDULES[schedule])
    assert error <= (PROMISE_EQUAL if kind == "same" else PROMISE_MANY) + floor


#: the Polar Express schedule (Amsel, Persson, Musco, Gower 2025) with its safety factor of 1.01
POLAR = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in
         ((8.28721201814563, -23.595886519098837, 17.300387312530933),
          (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
          (3.9486908534822946, -2.908902115962949, 0.5518191394370137),
          (3.3184196573706015, -2.488488024314874, 0.51004894012372),
          (2.300652019954817, -1.6689039845747493, 0.4188073119525673),
          (1.891301407787398, -1.2679958271945868, 0.37680408948524835),
          (1.8750014808534479, -1.2500016453999487, 0.3750001645474248))] + [(1.875, -1.25, 0.375)]


def code(coefficients):
    o = muon._options(0.0, False, len(coefficients), coefficients, 1e-7)
    return flce.lib().flce_orthogonalize((binding.Matrix * 1)((0x1000, 0x2000, 8, 8, 0)), 1, ctypes.byref(o), 0x100000,
                                         0, None)


def test_singular_values_of_up_to_2_1_are_taken():
    """(4: all is well but the workspace's size.)"""
    for n in range(1, 9):
        assert code(POLAR[:n]) == 4
    assert code([(2.05, 0.0, 0.0)]) == 4 and code([(2.1, 0.0, 0.0)]) == 1
    assert code([(2.05, 0.0, 0.0), (0.9, 0.0, 0.0)]) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["noise", "strong", "same", "rank8", "rank1", "decay"])
@pytest.mark.parametrize("r,c", [(64, 200), (128, 128), (300, 777), (640, 400)])
@pytest.mark.parametrize("steps", [1, 5, 8, 16])
def test_steep_first_steps(r, c, kind, steps):
    error, floor = off(matrix(r, c, kind).cuda(), POLAR[:steps] + POLAR[-1:] * (steps - 8))
    assert error <= (PROMISE if min(r, c) <= 128 else PROMISE_EQUAL) + floor


@pytest.mark.gpu
@pytest.mark.parametrize("r,c", [(48, 96), (200, 300)])
@pytest.mark.parametrize("second", [(0.9, -0.06, 0.01), (0.9, 0.06, -0.01), (0.5, 0.06, 0.01)])
def test_the_largest_singular_value_and_shift(r, c, second):
    """One direction at 2.05, where A and its shifted diagonal are largest."""
    u = with_values(r, c, [1.0] + [1e-3] * (min(r, c) - 1)).cuda()
    error, floor = off(u, [(2.05, 0.0, 0.0), second])
    assert error <= (PROMISE if min(r, c) <= 128 else PROMISE_EQUAL) + floor


@pytest.mark.gpu
def test_many_steps_captured_and_replayed():
    """Small matrices' further reads of X and larger ones' pairs in a graph, with a workspace of any content."""
    xs = [matrix(r, c, "strong", r).cuda() for r, c in ((200, 300), (40, 60), (128, 640))]
    table = (binding.Matrix * 3)(*((1, 1, *x.shape, 1) for x in xs))
    ws = torch.full((flce.lib().flce_orthogonalize_workspace_bytes(table, 3),), 255, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x, dtype=torch.bfloat16) for x in xs]
    flce.orthogonalize(xs, steps=11, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        flce.orthogonalize(xs, steps=11, out=out, ws=ws)
    for k in range(3):
        for x in xs:
            x.copy_(matrix(*x.shape, "rank8", k))
        graph.replay()
        for y, z in zip(out, flce.orthogonalize(xs, steps=11)):
            assert torch.equal(y, z)
    assert flce.read_device_status(ws) == 0
