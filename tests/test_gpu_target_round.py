"""The target's calls together (examples/target_round.py): prompts, rounds, shortened caches.

After some rounds every sequence's cache must hold exactly its kept tokens' keys and values, and
the target's logits for its last token, computed through the cache, must be those of the model
run over the whole sequence in 64 bits on the cached keys and values."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from examples.target_round import Rounds, ToyTarget
from tests._paged import HALF, quantise64, pow2

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


@pytest.mark.parametrize("e4m3", [False, True])
def test_rounds_keep_what_they_accepted(e4m3):
    m = ToyTarget(vocab=200)
    prompts = [[5] * 1, list(range(60)), list(range(100, 190)), [7, 9]]
    r = Rounds(m, prompts, gamma=3, e4m3=e4m3)
    for _ in range(6):
        t = r.round()
        assert bool((t[:, 0] >= 0).all())  # every round emits a token
    assert 0 < r.accepted < 6 * 3 * len(prompts)  # some drafts were kept, some forgotten
    k, v, start = r.cached()
    for b, tokens in enumerate(r.tokens):
        n = int(r.kv_len[b])
        assert n == len(tokens) - 1  # all but the last, which the next chunk begins with
        assert int(r.last[b]) == tokens[-1]
        x = m.embed[torch.tensor(tokens[:-1], device="cuda")]
        qkv = (x.double() @ m.w_qkv.double()).view(n, -1, m.head_dim)
        for got, at in ((k, m.heads), (v, m.heads + m.kv_heads)):
            want = qkv[:, at:at + m.kv_heads]
            # fp32 sums of 512 products (2^-15 of their size at most), then bf16
            size = (x.double().abs() @ m.w_qkv.double().abs()).view(n, -1, m.head_dim)
            tol = HALF[torch.bfloat16] * want.abs() + size[:, at:at + m.kv_heads] * 2.0 ** -15
            if e4m3:  # half a code more, or half the row's smallest step (twice it where the
                # row's largest value sits on the border of the next scale)
                step = pow2(quantise64(want)[1].int() - 127)[..., None] * 2.0 ** -9
                tol = tol * (1 + 2.0 ** -4) + torch.maximum(want.abs() * 2.0 ** -4, step)
            assert bool(((got[start[b]:start[b + 1]].double() - want).abs() <= tol).all())
    # one more chunk, of the last tokens alone, against the definition on the cached k and v
    B = len(prompts)
    q_start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    r.kv_len += 1
    x = m.embed[r.last]
    qkv = (x @ m.w_qkv).view(B, -1, m.head_dim)
    q, nk, nv = qkv.split([m.heads, m.kv_heads, m.kv_heads], dim=1)
    sv.spec_kv_append(r.cache, nk, nv, r.table, q_start, r.kv_len)
    out = sv.spec_chunk_attention(q, r.cache, r.table, q_start, r.kv_len)["out"]
    k, v, start = r.cached()
    G = m.heads // m.kv_heads
    for b in range(B):
        kb, vb = (t[start[b]:start[b + 1]].double() for t in (k, v))
        s = torch.einsum("hgd,lhd->hgl", q[b].double().view(m.kv_heads, G, -1), kb) * m.head_dim ** -0.5
        p = torch.softmax(s, -1)
        o = torch.einsum("hgl,lhd->hgd", p, vb)
        mass = torch.einsum("hgl,lhd->hgd", p, vb.abs())
        # p and the output rounded to bf16 once each; the scores' sums in fp32 move a
        # weight by 2 (64 + 8) S 2^-24 < 2^-12 for any |q||k| sum S < 20
        tol = HALF[torch.bfloat16] * (o.abs() + 1.01 * mass) + mass * 2.0 ** -12
        assert bool(((out[b].double().view_as(o) - o).abs() <= tol).all())


def test_the_example_runs(capsys, monkeypatch):
    import examples.target_round as ex
    monkeypatch.setattr("sys.argv", ["target_round.py", "--rounds", "2", "--e4m3"])
    ex.main()
    assert "drafts accepted" in capsys.readouterr().out


def test_a_full_cache_ends_the_rounds():
    """The last round that fits leaves its tokens in the cache; the next is refused."""
    m = ToyTarget(vocab=50)
    with pytest.raises(ValueError):
        Rounds(m, [[1] * 34, [2]], gamma=3, room=32)
    r = Rounds(m, [[1] * 25, [2]], gamma=3, room=32)
    done = 0
    while len(r.tokens[0]) + 3 <= 32:
        r.round()
        done += 1
    assert done and int(r.kv_len.max()) <= 32
    before = [list(t) for t in r.tokens]
    with pytest.raises(ValueError):
        r.round()
    assert r.tokens == before and r.cached()[2][-1] == sum(len(t) - 1 for t in before)
