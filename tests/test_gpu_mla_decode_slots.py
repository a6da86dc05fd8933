"""dsa_mla_decode over caches whose last page is cut short (n_slots no multiple of
the block or of 16): every slot that there is counts, those behind it are left out
and flagged if the sequence has tokens there.  Bounds as in test_gpu_mla_decode."""
import pytest
import torch

from tests.test_gpu_mla_decode import SCALE, check, inputs, tree

pytestmark = pytest.mark.gpu

# rows a request choose the form: up to 16, up to 32, up to 128, more
FORMS = [(16, 1), (32, 1), (128, 1), (64, 3)]


def cut_short(H, drafts, lens, block, n_off, page, seed):
    """Request 0's page `page` is the cache's last, which loses n_off slots."""
    args = list(inputs([drafts] * len(lens), lens, H, 2, 1, block, seed=seed))
    cache, table = args[1], args[2]
    last = cache.shape[1] // block - 1
    for s in range(2):
        at = (table[s] == last).nonzero()[0].tolist()
        table[s][tuple(at)], table[s, 0, page] = int(table[s, 0, page]), last
    args[1] = cache[:, :cache.shape[1] - n_off].contiguous()
    return args


@pytest.mark.parametrize("H,drafts", FORMS)
@pytest.mark.parametrize("block,n_off", [(64, 28), (64, 1), (64, 63), (16, 5), (32, 17), (192, 70), (128, 127)])
def test_a_sequence_that_ends_in_the_last_page(H, drafts, block, n_off):
    """Its tokens there all lie inside the cache, up to the last slot."""
    import dsa_sparse_indexer_gb300 as dsa
    page = 300 // block
    lens = [2 * (page * block + block - n_off), 90]
    args = cut_short(H, drafts, lens, block, n_off, page, seed=block + n_off)
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_decode(*args, SCALE, err_flags=err)
    assert int(err) == 0
    check(args, SCALE, None, out, lse2)


@pytest.mark.parametrize("H,drafts", FORMS)
@pytest.mark.parametrize("block,n_off", [(64, 28), (64, 16), (16, 5), (32, 17), (192, 70)])
def test_a_sequence_that_goes_on_behind_the_last_slot(H, drafts, block, n_off):
    """In its middle a page is cut short: the tokens behind the last slot alone are
    left out, with a chain and with a tree whose drafts lie elsewhere."""
    import dsa_sparse_indexer_gb300 as dsa
    args = cut_short(H, drafts, [900, 90], block, n_off, 100 // block, seed=block + n_off)
    for mask in (None, tree([drafts] * 2)):
        err = dsa.new_error_flags("cuda")
        out, lse2 = dsa.mla_decode(*args, SCALE, tree_mask=mask, err_flags=err)
        assert int(err) == dsa.DSA_FLAG_BOUNDS
        check(args, SCALE, mask, out, lse2)


@pytest.mark.parametrize("H,drafts", FORMS)
def test_a_cache_of_less_than_16_slots(H, drafts):
    import dsa_sparse_indexer_gb300 as dsa
    args = list(inputs([drafts], [11], H, 1, 1, 64, seed=3))
    args[1] = args[1][:, :11].contiguous()
    err = dsa.new_error_flags("cuda")
    out, lse2 = dsa.mla_decode(*args, SCALE, err_flags=err)
    assert int(err) == 0 and torch.isfinite(lse2).all()
    check(args, SCALE, None, out, lse2)
