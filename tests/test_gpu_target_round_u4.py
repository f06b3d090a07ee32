"""The example's rounds with rotary positions and a cache of 4 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from examples.target_round import Rounds, ToyTarget

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()
    flags = torch.backends.cuda.matmul
    was = flags.allow_bf16_reduced_precision_reduction
    flags.allow_bf16_reduced_precision_reduction = False  # the projections' sums in fp32
    yield
    flags.allow_bf16_reduced_precision_reduction = was


def test_the_example_runs(capsys, monkeypatch):
    import examples.target_round as ex
    for flags in (["--u4"], ["--rotary"], ["--u4", "--rotary"], ["--e4m3", "--rotary"]):
        monkeypatch.setattr("sys.argv", ["target_round.py", "--rounds", "2", *flags])
        ex.main()
        assert "drafts accepted" in capsys.readouterr().out


def test_rounds_keep_what_they_accepted():
    """Lengths after every round, and the cached rows against what the tokens' own rows become: the
    projections are the same products in other shapes, bf16 rows one rounding apart at most (2^-7 of
    the value; sums of 512 products move it by 2^-15 of their size); a turn adds two such rows; a
    code half a step, and the row's largest and smallest value, which set the step, move its zero
    and 15 steps by as much as they move themselves, with the step's and the zero's rounding to
    bf16, half a 2^-7 of each."""
    m = ToyTarget(vocab=200, rotary=512)
    prompts = [[5] * 1, list(range(60)), list(range(100, 190)), [7, 9]]
    r = Rounds(m, prompts, gamma=3, u4=True)
    for _ in range(6):
        assert bool((r.round()[:, 0] >= 0).all())
    k, v, start = r.cached()
    for b, tokens in enumerate(r.tokens):
        n = int(r.kv_len[b])
        assert n == len(tokens) - 1 and int(r.last[b]) == tokens[-1]
        x = m.embed[torch.tensor(tokens[:-1], device="cuda")]
        rows = (x.double() @ m.w_qkv.double()).view(n, -1, m.head_dim)
        size = (x.double().abs() @ m.w_qkv.double().abs()).view(n, -1, m.head_dim)
        c, s = m.cos_sin[:n].double()[:, None].chunk(2, -1)
        for got, at, turned in ((k, m.heads, True), (v, m.heads + m.kv_heads, False)):
            want, off = rows[:, at:at + m.kv_heads], size[:, at:at + m.kv_heads] * 2.0 ** -15
            off = off + want.abs() * 2.0 ** -7
            if turned:
                (x0, x1), (d0, d1) = want.chunk(2, -1), off.chunk(2, -1)
                want = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
                off = torch.cat([d0 * c.abs() + d1 * s.abs(), d1 * c.abs() + d0 * s.abs()], -1)
            lo, hi = want.amin(-1, keepdim=True), want.amax(-1, keepdim=True)
            most, far = off.amax(-1, keepdim=True), torch.maximum(lo.abs(), hi.abs())
            step = (hi - lo + 2 * most + far * 2.0 ** -8) / 15
            # (the value that was read is rounded to bf16 as well)
            tol = (off + step * (0.5 + 15 * 2.0 ** -8) + 3 * most + far * 2.0 ** -7) * 1.01
            assert bool(((got[start[b]:start[b + 1]].double() - want).abs() <= tol).all())
