"""spec_verify_probs against the definition in exact integers."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


def reference(p, q, x, u):
    """Tokens, counts and flags by the definition: fp32 quotients and differences, sums as whole
    numbers of 2^-61."""
    p, q, u = (np.asarray(a, dtype=np.float32) for a in (p, q, u))
    B, G, V = q.shape
    tokens = np.full((B, G + 1), -1, dtype=np.int32)
    counts, flags = np.zeros(B, dtype=np.int32), np.zeros(B, dtype=np.int32)
    sane = lambda a: np.where((a >= 0) & (a <= 2), a, np.float32(0))  # noqa: E731
    for b in range(B):
        n = 0
        while n < G:
            t, f = int(x[b, n]), 0
            pt = qt = np.float32(0)
            if not 0 <= t < V:
                f |= sv.FLAG_BAD_TOKEN
            else:
                pt, qt = sane(p[b, n, t]), sane(q[b, n, t])
                if pt != p[b, n, t] or qt != q[b, n, t] or qt == 0:
                    f |= sv.FLAG_NONFINITE
            if not 0 <= u[b, n] < 1:
                f |= sv.FLAG_NONFINITE
            flags[b] |= f
            with np.errstate(divide="ignore", invalid="ignore"):
                if not u[b, n] <= pt / qt:
                    break
            tokens[b, n] = t
            n += 1
        pn = sane(p[b, n])
        odd = bool((pn != p[b, n]).any())
        w = pn
        if n < G:
            qn = sane(q[b, n])
            odd |= bool((qn != q[b, n]).any())
            w = np.maximum(np.float32(0), pn - qn)
            if not (w > 0).any():
                flags[b] |= sv.FLAG_RESIDUAL_FALLBACK
                w = pn
        if not (w > 0).any():
            flags[b] |= sv.FLAG_ZERO_MASS
        run = np.cumsum(np.rint(w.astype(np.float64) * 2.0 ** 61).astype(np.uint64))
        ub = float(u[b, G])
        if not 0 <= ub < 1:
            odd = True
            ub = float(np.float32(1) - np.float32(2.0 ** -24)) if ub >= 1 else 0.0
        target = int(Fraction(ub) * int(run[-1]))
        past = np.nonzero(run > np.uint64(target))[0]
        tokens[b, n] = past[0] if len(past) else 0
        flags[b] |= sv.FLAG_NONFINITE if odd else 0
        counts[b] = n
    return tokens, counts, flags


def make(B, G, V, dtype=torch.float32, seed=0, noise=0.5, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    zt = torch.randn((B, G + 1, V), generator=g, device="cuda") * spread
    zd = zt[:, :G] + torch.randn((B, G, V), generator=g, device="cuda") * noise
    p, q = torch.softmax(zt, -1).to(dtype), torch.softmax(zd, -1).to(dtype)
    x = torch.multinomial(q.reshape(-1, V).float(), 1, generator=g).reshape(B, G).int()
    u = torch.rand((B, G + 1), generator=g, device="cuda")
    return p.contiguous(), q.contiguous(), x, u


def check(p, q, x, u):
    o = sv.spec_verify_probs(p, q, x, u, want_flags=True)
    torch.cuda.synchronize()
    t, c, f = reference(p.float().cpu().numpy(), q.float().cpu().numpy(), x.cpu().numpy(),
                        u.cpu().numpy())
    np.testing.assert_array_equal(o["counts"].cpu().numpy(), c)
    np.testing.assert_array_equal(o["tokens"].cpu().numpy(), t)
    np.testing.assert_array_equal(o["flags"].cpu().numpy(), f)
    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,G,V", [(1, 1, 1), (3, 1, 2), (5, 4, 7), (64, 4, 1000), (1, 4, 32000),
                                   (2, 8, 32003), (200, 3, 4099), (7, 32, 513), (33, 2, 16384),
                                   (1, 2, 128256), (400, 1, 100)])
def test_rounds(B, G, V, dtype):
    for seed in range(3):
        check(*make(B, G, V, dtype, seed, noise=(0.1, 0.5, 2.0)[seed]))


def test_every_token_of_a_row_is_reached_at_its_border():
    """u on, just below and just above each border of the cumulative weights."""
    V = 64
    w = torch.tensor([(v * 7 % 5) / 128.0 for v in range(V)])  # some zero; sums exact
    w = w / 1.0
    total = float(w.sum())
    edges = (torch.cumsum(w, 0) / total).tolist()
    us = sorted({float(np.float32(e)) for e in edges[:-1]})
    us = [float(np.nextafter(np.float32(e), np.float32(s))) for e in us for s in (0, 1)] + us + [0.0]
    us = [e for e in us if 0 <= e < 1]
    B = len(us)
    p = w.expand(B, 2, V).contiguous().cuda()
    q = p[:, :1].contiguous()  # equal: every draft is accepted, the bonus row is drawn
    x = torch.full((B, 1), int(torch.nonzero(w)[0]), dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.5, e] for e in us], device="cuda")
    o = check(p, q, x, u)
    assert bool((w.cuda()[o["tokens"][:, 1].long()] > 0).all())


def test_one_entry_holds_everything():
    for V in (5, 4096, 70001):
        for at in (0, V // 2, V - 1):
            p = torch.zeros((2, 2, V), device="cuda")
            p[..., at] = 1.0
            q = torch.full((2, 1, V), 1.0 / V, device="cuda")
            x = torch.tensor([[at], [(at + 1) % V]], dtype=torch.int32, device="cuda")
            u = torch.tensor([[0.3, 0.999999], [0.3, 0.0]], device="cuda")
            o = check(p, q, x, u)
            assert o["tokens"][0, 1].item() == at and o["tokens"][1, 0].item() == at


def test_empty_residual_empty_row_and_tiny_weights():
    p, q, x, u = make(6, 2, 999, seed=4)
    q[0] = p[0, :2]          # equal rows ...
    x[0, 0], p[0, 0, 5] = 5, 0.0
    q[0, 0, 5] = 0.25        # ... whose draft is impossible for the target: residual empty
    p[1], p[2, 0] = 0.0, 0.0
    p[3] *= 1e-20            # weights near and below a unit
    q[3] *= 1e-20
    p[4, 2] = 1e-30
    u[4, :2] = 0.0
    check(p, q, x, u)


def test_values_that_are_no_probabilities():
    p, q, x, u = make(8, 2, 500, seed=5)
    p[0, :, 3], p[1, :, 4], p[2, :, 5], q[3, :, 6] = float("nan"), float("inf"), -0.5, float("nan")
    x[4, 0], x[5, 1] = -1, 500
    u[6, 2], u[7, 2] = 1.0, float("nan")
    check(p, q, x, u)
    u[6, 0], u[7, 0] = float("nan"), -1.0
    check(p, q, x, u)


def test_distribution_of_the_emitted_token():
    """p = (0.6, 0.3, 0.1), q = (0.2, 0.5, 0.3): the first emitted token follows p."""
    n = 200000
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    p = torch.tensor([0.6, 0.3, 0.1], device="cuda").expand(n, 2, 3).contiguous()
    q = torch.tensor([0.2, 0.5, 0.3], device="cuda").expand(n, 1, 3).contiguous()
    x = torch.multinomial(q[:, 0], 1, generator=g).int()
    u = torch.rand((n, 2), generator=g, device="cuda")
    t = sv.spec_verify_probs(p, q, x, u)["tokens"][:, 0]
    got = torch.bincount(t.long(), minlength=3).double() / n
    want = torch.tensor([0.6, 0.3, 0.1], dtype=torch.float64, device="cuda")
    assert bool(((got - want).abs() < 5 * torch.sqrt(want * (1 - want) / n)).all())


def test_another_stream_and_a_graph():
    p, q, x, u = make(16, 4, 5000)
    want = sv.spec_verify_probs(p, q, x, u)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = sv.spec_verify_probs(p, q, x, u)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sv.spec_verify_probs(p, q, x, u, out=out)
    s.synchronize()
    assert torch.equal(out["tokens"], want["tokens"])
    u.copy_(torch.rand_like(u))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["tokens"], sv.spec_verify_probs(p, q, x, u)["tokens"])


def test_refusals_of_the_binding():
    p, q, x, u = make(2, 2, 50)
    with pytest.raises(TypeError):
        sv.spec_verify_probs(p.half(), q.half(), x, u)
    with pytest.raises(TypeError):
        sv.spec_verify_probs(p, q, x.long(), u)
    with pytest.raises(TypeError):
        sv.spec_verify_probs(p, q, x, u.double())
    with pytest.raises(ValueError):
        sv.spec_verify_probs(p, q, x, u[:, :2])


def test_uniforms_of_the_accept_tests_are_compared_as_they_stand():
    """p/q = 1.25: 1.2 accepts, 1.5 rejects, NaN rejects, -3 accepts; each is flagged.  Behind the
    first rejection nothing is looked at."""
    p = torch.tensor([0.5, 0.5], device="cuda").expand(5, 3, 2).contiguous()
    q = torch.tensor([0.4, 0.6], device="cuda").expand(5, 2, 2).contiguous()
    x = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    u = torch.full((5, 3), 0.5, device="cuda")
    u[:4, 0] = torch.tensor([1.2, 1.5, float("nan"), -3.0])
    x[4, 0], u[4, 0], u[4, 1] = 1, 0.9, float("nan")  # 0.9 > 0.5 / 0.6
    o = check(p, q, x, u)
    assert o["counts"].tolist() == [2, 0, 0, 2, 0]
    assert o["flags"].tolist() == [sv.FLAG_NONFINITE] * 4 + [0]
