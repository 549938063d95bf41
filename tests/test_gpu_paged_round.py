"""The calls of a round run together on a paged cache: greedy speculative decoding of the example
emits what decoding token by token does, whatever was drafted, and every page is accounted for."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_matches_decoding_token_by_token():
    import paged_round
    got = paged_round.main(rounds=10)
    assert all(len(g) >= 10 for g in got)


@pytest.mark.parametrize("page,gamma", [(1, 3), (5, 7), (64, 1)])
def test_rounds_keep_the_pool_whole(page, gamma):
    import paged_round
    m = paged_round.Model(seed=3)
    prompts = [[1, 2, 3, 4, 5, 6, 7], [8, 9], [10]]
    s = paged_round.Rounds(m, prompts, gamma=gamma, page=page, blocks=300)
    s.prefill()
    for i in range(6):
        s.round(seed=i)
    torch.cuda.synchronize()
    head, count = s.free_state.tolist()
    ring, held = s.free_ring.tolist(), s.held.tolist()
    pages = [ring[(head + i) % 300] for i in range(count)]
    pages += [int(x) for b in range(3) for x in s.table[b, :held[b]]]
    assert sorted(pages) == list(range(300))
    want = paged_round.token_by_token(m, prompts, int((s.history_len - s.prompt_len).max()))
    for b in range(3):
        p, n = int(s.prompt_len[b]), int(s.history_len[b])
        assert s.history[b, p:n].tolist() == want[b][:n - p]
