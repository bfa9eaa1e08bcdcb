"""append and evict once more, with every byte that is no code compared bit
for bit: the scales, the gaps between the pages and the pages' ends."""
import pytest
import torch

import test_kv_gpu as base
from kv_same import assert_same_arena

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ac():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import arena_compaction_amd
    return arena_compaction_amd


@pytest.fixture(autouse=True)
def bit_for_bit(monkeypatch):
    monkeypatch.setattr(base, "same", assert_same_arena)


test_append = base.test_append
test_append_layouts = base.test_append_layouts
test_append_odd_numbers = base.test_append_odd_numbers
test_append_refuses_bad_pages = base.test_append_refuses_bad_pages
test_evict = base.test_evict
test_evict_ties_and_safe_tokens = base.test_evict_ties_and_safe_tokens
test_evict_odd_weights = base.test_evict_odd_weights
test_evict_long = base.test_evict_long
test_evict_longer_rows = base.test_evict_longer_rows
test_evict_longer_rows_bad_pages = base.test_evict_longer_rows_bad_pages
test_evict_leaves_bad_sequences_alone = base.test_evict_leaves_bad_sequences_alone
test_offsets_past_32_bits = base.test_offsets_past_32_bits
