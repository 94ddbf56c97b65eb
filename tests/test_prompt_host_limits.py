"""Further host-side checks of the KDA prefill (no GPU needed)."""
import retrieve_store_chunk_amd as hkv
from tests.test_ops_host import layout
from tests.test_prompt_host import prefill_args


def test_calls_of_many_blocks_have_room_to_count_them():
    """8 bytes for each of the pool's blocks, where the call's rows hold more than 24
    whole blocks."""
    lay = layout()
    n, blocks = lay.info["block_size"], lay.info["num_blocks"]

    def size(tokens, **kw):
        return lay.kda_prefill_workspace(prefill_args(n_tokens=tokens, max_seq_tokens=tokens, **kw))

    few, many = size(25 * n - 1), size(25 * n)
    assert many - few >= 8 * blocks > 0
    assert size(25 * n - 1, n_seqs=4096) < size(25 * n, n_seqs=4096)
    assert size(1 << 20) == many
    assert hkv.status_of(lay.kda_prefill, 1 << 40, prefill_args(n_tokens=25 * n, max_seq_tokens=25 * n),
                         0x7F0000000000, few, 0) == hkv.HKV_E_WORKSPACE
