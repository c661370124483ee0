"""GPU: the optimizer at the edges of what a program does with it.

u = 2^-24, a rounding of single precision."""
import numpy as np
import pytest
import torch

from gpu_util import host
from oracle import layer

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24


def small(bits=32, master=False, n=600):
    kind = torch.bfloat16 if master else torch.float32
    params = [torch.full((n,), 0.5, device="cuda", dtype=kind), torch.zeros(7, device="cuda", dtype=kind)]
    grads = [torch.full((n,), 1e-2, device="cuda"), torch.ones(7, device="cuda")]
    return ap.AdamW(params, grads, master=master, state_bits=bits)


def move_param(o):
    o.params[1].data = o.params[1].data.clone()


def move_master(o):
    o.master[0].data = o.master[0].data.clone()


def load_state(o):
    o.state.update({n: t.clone() for n, t in o.state.items()})


def replace_scale(o):
    o.state["v_scale"] = torch.zeros(1, device="cuda")


def free_state(o):
    o.state["m"].untyped_storage().resize_(0)


@pytest.mark.parametrize("move", [move_param, move_master, load_state, replace_scale, free_state])
def test_tensors_that_moved_are_refused(move):
    """A step writes where its tensors were when the optimizer was made, so it refuses those that are elsewhere now."""
    o = small(8, True)
    o.step()
    kept = [t.clone() for t in o.params + o.master]
    move(o)
    n0 = ap.launch_count()
    for call in (o.step, o.moments):
        with pytest.raises(ValueError, match="moved"):
            call()
    assert ap.launch_count() == n0
    assert all(torch.equal(a, b) for a, b in zip(kept, o.params + o.master))


def test_gradients_that_moved_are_refused_until_bound_again():
    o = small()
    o.grads[0].data = torch.full((600,), -1e-2, device="cuda")
    n0 = ap.launch_count()
    for call in (o.step, o.grad_norm):
        with pytest.raises(ValueError, match="bind"):
            call()
    assert ap.launch_count() == n0
    o.bind(o.grads)
    before = float(o.params[0][0])
    o.step()
    assert float(o.params[0][0]) > before  # down the new gradient


def test_loaded_state_is_copied_in_or_given_anew():
    a, b = small(8), small(8)
    a.step()
    for name, t in b.state.items():
        t.copy_(a.state[name])
    for x, y in zip(a.params, b.params):
        y.copy_(x)
    c = ap.AdamW([p.clone() for p in a.params], a.grads, state_bits=8, state={n: t.clone() for n, t in a.state.items()})
    for o in (a, b, c):
        o.step()
    for o in (b, c):
        assert all(torch.equal(x, y) for x, y in zip(a.params + list(a.state.values()), o.params + list(o.state.values())))
    assert host(a.state["step"]).tolist() == [2, 0] and np.isfinite(host(a.params[0])).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_skip_word_that_changes_during_the_call_is_read_once(bits):
    """441 tensors are two launches.  Another stream flips the word all the while: a step is taken whole or not at all, and
    the work word is 0 after it."""
    n = 40_000
    params = [torch.ones(n, device="cuda") for _ in range(441)]
    o = ap.AdamW(params, [torch.ones(n, device="cuda") for _ in range(441)], weight_decay=0.0, state_bits=bits)
    word, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    steps, ends = 0, torch.stack([p[i] for p in params for i in (0, -1)])
    torch.cuda.synchronize()
    for _ in range(30):
        for q in range(40):
            with torch.cuda.stream(side):
                word.fill_(q & 1)
            if q == 20:
                o.step(skip=word)
        torch.cuda.synchronize()
        now, work = host(o.state["step"]).tolist()
        was, ends = ends, torch.stack([p[i] for p in params for i in (0, -1)])
        assert work == 0 and now - steps in (0, 1)
        moved = ends != was  # (a step of gradients of 1 moves each element by about lr)
        assert bool(moved.all()) if now > steps else not bool(moved.any())
        steps = now


def test_a_step_after_a_skipped_one_counts_from_the_start():
    o, word = small(), torch.ones(1, dtype=torch.int32, device="cuda")
    for skip, steps in ((word, 0), (None, 1), (word, 1), (word, 1), (torch.zeros_like(word), 2), (None, 3)):
        o.step(skip=skip)
        assert host(o.state["step"]).tolist() == [steps, 0]
    o.step(scale=torch.full((1,), float("nan"), device="cuda"), skip=torch.zeros_like(word))
    assert host(o.state["step"]).tolist() == [3, 0]


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lr,decay", [(1e-2, 0.1), (1e-5, 0.01), (3e-6, 0.01), (2e-6, 0.01)])
def test_small_decays_are_whole(kind, lr, decay):
    """The end of a schedule, lr * decay down to 2e-8: over many elements the change is the formula's.  Parameters in [1, 2)
    round to multiples of 2 u: by u at the most, either way alike, as the changes (of deviation lr, 16 such steps and more)
    spread over many.  So the mean of n has a deviation of u / sqrt(3 n); six of them, and 64 u of the mean change (of lr, rate,
    product and quotient).  The decay is 0.5 u and more."""
    n = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.rand(n, generator=g, device="cuda") + 1.0
    state = {"m": torch.randn(n, generator=g, device="cuda"), "v": torch.ones(n, device="cuda"),
             "step": torch.tensor([10 ** 6, 0], dtype=torch.int32, device="cuda")}
    grad = torch.randn(n, generator=g, device="cuda")
    before, m, v = p.double(), state["m"].double(), state["v"].double()
    o = ap.AdamW([p.to(kind)], [grad], lr=lr, weight_decay=decay, state=state, master=[p] if kind == torch.bfloat16 else None)
    o.step()
    after = (o.master or o.params)[0].double()
    m, v = 0.9 * m + 0.1 * grad.double(), 0.999 * v + 0.001 * grad.double() ** 2
    change = -lr * decay * before - lr * m / (v.sqrt() + 1e-8)  # (the corrections are 1 by then)
    off = float((after - before - change).mean())
    assert abs(off) <= 6 * U / (3 * n) ** 0.5 + 64 * U * abs(float(change.mean()))


@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_squares_below_the_normal_numbers_have_roots(eps):
    """v near 1e-40: the change is the formula's, for eps = 0 too.  v = b2 v rounds by 2^-150 (of 1e-40: 7e-6 u', half of that
    in its root), the rest by 32 u."""
    n = 1024
    state = {"m": torch.linspace(-1e-22, 1e-22, n, device="cuda"), "v": torch.linspace(1e-40, 3e-40, n, device="cuda"),
             "step": torch.tensor([10 ** 6, 0], dtype=torch.int32, device="cuda")}
    m, v = state["m"].double() * 0.9, state["v"].double() * 0.999
    o = ap.AdamW([torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")], lr=1.0, eps=eps, weight_decay=0.0, state=state)
    o.step()
    want = -m / (v.sqrt() + eps)
    assert bool((o.state["v"] > 0).all())
    assert bool(((o.params[0].double() - want).abs() <= (0.5 * 2.0 ** -150 / 1e-40 + 32 * U) * want.abs()).all())


def test_codes_of_positive_squares_are_positive():
    """Gradients of 1e-20 to 1e-19: (1 - b2) g^2 is 1e-43 and more, below the normal numbers but positive."""
    n = 512
    o = ap.AdamW([torch.zeros(n, device="cuda")], [torch.logspace(-20, -19, n, device="cuda")], lr=1.0, eps=0.0, state_bits=8)
    o.step()
    assert bool((o.state["v"] > 0).all()) and bool(torch.isfinite(o.params[0]).all())
    m, v = o.moments()
    assert bool((v > 0).all()) and bool((o.params[0] < 0).all())


@pytest.mark.parametrize("ratio", [1e-2, 1e-3, 1e-4, 1e-5])
def test_small_moments_in_codes_keep_their_size(ratio):
    """Elements far below their block's largest, of one gradient: coded moments rounded by values keep the mean.  A code's
    expectation is the value, to half of 2^-17 of a step between codes (below the value itself, but for codes near 0: of
    2^-17 scales, 7.6e-6 of m = 0.16 scales); the mean of n elements is off by its standard deviation, six of them.  v of
    1e-5 lies below its scale's first code, which it is kept at."""
    n, steps = 1 << 20, 60
    grad = torch.full((n,), ratio, device="cuda")
    grad[::256] = 1.0
    o = ap.AdamW([torch.zeros(n, device="cuda")], [grad], betas=(0.9, 0.95), state_bits=8, rounding="values", seed=5)
    for _ in range(steps):
        o.step()
    for name, moment, want, b in (("m", o.moments()[0], ratio, 0.9), ("v", o.moments()[1], ratio ** 2, 0.95)):
        x = moment.view(-1, 256)[:, 1:].double()
        want *= 1 - b ** steps
        if name == "v" and ratio == 1e-5:
            assert bool((o.state["v"].view(-1, 256)[:, 1:] == 1).all())
            continue
        assert abs(float(x.mean()) - want) <= 6 * float(x.std()) / x.numel() ** 0.5 + (2e-4 + 64 * U) * want


@pytest.mark.parametrize("rounding", ["codes", "values"])
def test_codes_are_the_documented_ones(rounding):
    """Of a first step, whose moments are (1 - b) g and (1 - b) g^2: x = |m| / m_scale takes 8 u of itself, and a code
    rises with x.  The place between two values takes 8 u more of the values, which is a fraction of the step between
    them of 8 u x / (2 c + 1) < 8 u 128 at most (v: half its power's): covered by 1024 u of x."""
    n = 256 * 64 + 100
    g = torch.Generator(device="cuda").manual_seed(9)
    grad = torch.randn(n, generator=g, device="cuda") * torch.logspace(-4, 0, n, device="cuda")[torch.randperm(n, generator=g, device="cuda")]
    grad[:256] = 0.0
    o = ap.AdamW([torch.zeros(n, device="cuda")], [grad], betas=(0.9, 0.95), state_bits=8, rounding=rounding, seed=7)
    o.step()
    low, high = layer.adamw_noise(7, 1, 0, n)
    gf = host(grad).astype(np.float64)
    for name, x, top, r, power in (("m", np.abs(gf) * 0.1, 127, low, 1), ("v", np.abs(gf) * np.sqrt(0.05), 255, high, 2)):
        scale = np.repeat(layer.block_max(x) / top ** 2, 256)[:n]
        on = scale > 0
        y = np.where(on, x / np.where(on, scale, 1.0), 0.0)
        code = np.abs(host(o.state[name])[:n].astype(np.int64))
        lo, hi = (layer.adamw_codes(y * (1 + d), r + d, top, power, rounding) for d in (-1024 * U, 1024 * U))
        if name == "v":
            lo, hi = np.maximum(lo, y > 0), np.maximum(hi, y > 0)
        if rounding == "values":  # (r is compared with the place, which falls with it)
            lo = np.minimum(lo, layer.adamw_codes(y * (1 - 1024 * U), r + 1024 * U, top, power, rounding))
            hi = np.maximum(hi, layer.adamw_codes(y * (1 + 1024 * U), r - 1024 * U, top, power, rounding))
            if name == "v":
                lo = np.maximum(lo, y > 0)
        assert np.all((code >= lo) & (code <= hi))
        assert (lo == hi).mean() > 0.98  # (the bounds leave few codes open)
        assert not code[~on].any()


def test_rounding_by_values_is_seeded_and_repeats():
    def run(seed):
        o = ap.AdamW([torch.zeros(1000, device="cuda")], [torch.linspace(-1, 1, 1000, device="cuda")], state_bits=8, rounding="values",
                     seed=seed)
        for _ in range(3):
            o.step()
        return list(o.state.values()) + o.params
    a, b, c = run(1), run(1), run(2)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not torch.equal(a[1], c[1])


@pytest.mark.parametrize("rounding", ["codes", "values"])
def test_captured_steps_read_the_skip_word_at_each_replay(rounding):
    def make():
        g = torch.Generator(device="cuda").manual_seed(2)
        params = [torch.randn(n, generator=g, device="cuda").bfloat16() for n in (700, 3, 5000)]
        grads = [torch.randn(n, generator=g, device="cuda") for n in (700, 3, 5000)]
        return ap.AdamW(params, grads, master=True, state_bits=8, rounding=rounding, seed=3)
    a, b = make(), make()
    word, side = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        a.step(skip=word)
    steps = 0
    for skip in (0, 1, 1, 0, 2 ** 31 - 1, 0):
        word.fill_(skip)
        graph.replay()
        b.step(skip=word)
        steps += skip == 0
        assert host(a.state["step"]).tolist() == host(b.state["step"]).tolist() == [steps, 0]
    for x, y in zip(a.params + a.master + list(a.state.values()), b.params + b.master + list(b.state.values())):
        assert torch.equal(x, y)
