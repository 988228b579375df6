"""The forward calls in a workspace of the largest batch's size: smaller batches, and the chunks
of a long one, stay within it and give what they give in a workspace with room to spare."""
import numpy as np
import pytest
import torch

import engram_gram_conditional_gb300 as eg
import synth
from helpers import from_dev, prefill_windows, setup_workload, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from engram_gram_conditional_gb300 import build

    build.build()
    assert torch.cuda.is_available()


def check(s, most, batches, staged):
    ctx = s.model.ctx
    need = (eg.engram_forward_staged_workspace_bytes if staged else eg.engram_workspace_bytes)(ctx, most)
    guarded = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    plenty = torch.full((1 << 28,), 0xA5, dtype=torch.uint8, device="cuda")
    win, _, _ = prefill_windows(s, 1, most)
    hidden = synth.hidden_bf16(s.w, most)
    for T in batches:
        out = []
        for ws in (guarded[256:], plenty):
            h, g = to_dev(hidden[:T]), torch.full((T, s.w.hc), float("nan"), device="cuda")
            (eg.engram_forward_staged if staged else eg.engram_forward)(ctx, 0, to_dev(win[:T]), T, h, ws, g)
            eg.engram_sync(ctx)
            out.append((from_dev(h, np.uint16), g.cpu().numpy()))
        assert np.array_equal(out[0][0], out[1][0]) and np.array_equal(out[0][1], out[1][1]), T
        assert not np.array_equal(out[0][0], hidden[:T])
        assert (guarded[:256] == 0xA5).all() and (guarded[256 + need:] == 0xA5).all(), T


def test_a_long_batch_of_a_small_layer_runs_its_chunks_within_the_workspace():
    # 2 branches x 256: 13,200 tokens fill the GPU, a chunk of at most 6,144 does not
    s = setup_workload("tiny")
    check(s, 13_200, (1, 300, 6000, 13_200), staged=True)
    s.close()


@pytest.mark.parametrize("staged", [False, True])
def test_smaller_batches_in_the_workspace_of_the_largest(staged):
    # 24 rows of 256: a small batch splits K, or parks stream-K pieces
    s = setup_workload("tiny", layers=[0], heads=8, row_dim=256, hc=1, d=256)
    check(s, 20_000, (1, 128, 129, 1000, 20_000), staged=staged)
    s.close()
