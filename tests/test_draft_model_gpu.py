"""The example that uses the language-model row operators together: a draft
model learns from stored top logits, and its drafts are accepted more often."""
import pytest

import shape_adaptive_tile_gb300 as sat

pytestmark = pytest.mark.gpu


def test_the_draft_model_learns_and_its_drafts_are_accepted():
    sat.build()
    from examples import draft_model
    losses, before, after = draft_model.main(vocab=1024, width=256, batch=512, k=16, steps=40, drafts=3)
    assert losses[-1] < 0.8 * losses[0]
    assert after > before
