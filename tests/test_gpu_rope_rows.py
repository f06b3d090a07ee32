"""spec_kv_append_rope where an entry of q_start is bad: flags, queries and keys of every sequence,
those beside the bad entry and those that it must not touch."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_21_gb300 as sv
from tests._paged import E4M3
from tests._paged_u4 import BF, U4, codes_of, packed
from tests.test_gpu_rope import make, projection, rotate, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load()


@pytest.mark.parametrize("cache", [BF, E4M3, U4])
@pytest.mark.parametrize("start", [[0, 7, 4, 9], [0, -1, 9, 9], [0, 4, 100, 9], [0, 4, 4, 9], [0, 4, 3, 9],
                                   [0, 9, 9, 9], [3, 4, 6, 6], [2 ** 30, 4, 7, 9], [0, 4, 7, -2 ** 31]])
def test_a_bad_start_leaves_the_others_alone(start, cache):
    """A sequence is sound where 0 <= start[b] <= start[b + 1] <= total; its rows are rotated at its
    own positions (a row of two sound ones, at the positions of either)."""
    total, lens = 9, [20, 30, 40]
    c = make([(4, 20), (3, 30), (2, 40)], cache)
    q, k, v = projection(c, 4)
    rope = table_of(64, 64)
    c.cache.k.view(torch.uint8).fill_(7)
    held = c.cache.k.view(torch.uint8).clone()
    out = {"q": torch.full((total, 4, c.D), 5.0, dtype=BF, device="cuda")}
    o = sv.spec_kv_append_rope(c.cache, k, v, c.table, torch.tensor(start, dtype=torch.int32, device="cuda"),
                               c.len, rope, q=q, out=out, want_flags=True)
    sound = [0 <= start[b] <= start[b + 1] <= total for b in range(3)]
    assert o["flags"].tolist() == [0 if x else sv.FLAG_BAD_LENGTH for x in sound]
    written = {}
    for t in range(total):
        owners = [(b, lens[b] - (start[b + 1] - t)) for b in range(3) if sound[b] and start[b] <= t < start[b + 1]]
        wants = [rotate(q[t:t + 1].float(), rope[pos][None], False).to(BF)[0] for _, pos in owners]
        if not owners:
            assert bool((o["q"][t] == 5.0).all()), t
            continue
        hit = [i for i, w in enumerate(wants) if torch.equal(o["q"][t], w)]
        assert hit, t
        b, pos = owners[hit[0]]
        written[c.owned[b][pos // c.ps], pos % c.ps] = rotate(k[t:t + 1].float(), rope[pos][None], False)[0]
    got = c.cache.k.view(torch.uint8)
    for page in range(c.pages):
        for slot in range(c.ps):
            x = got[page, :, slot]
            if (page, slot) not in written:
                assert torch.equal(x, held[page, :, slot]), (page, slot)
            elif cache == U4:
                assert torch.equal(x, packed(codes_of(written[page, slot])[0]))
            elif cache == BF:
                assert torch.equal(x.contiguous().view(BF), written[page, slot].to(BF))
            else:
                assert not torch.equal(x, held[page, :, slot])
