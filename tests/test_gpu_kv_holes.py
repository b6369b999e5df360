"""Missing pages under gdn_kv_attention, page by page: of every size, in both forms, behind windows
and in units that are split between CTAs.  Nothing of a page that is none is seen.  Bounds as in
test_gpu_kv_attention.py."""
import pytest

from test_gpu_kv_attention import check

pytestmark = pytest.mark.gpu
PAGES = [16, 32, 64, 128, 256]


def without(gone):
    def change(q, cache, table, kv):
        table[0, gone] = -1 if gone % 2 else cache.shape[0]
    return change


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("new,window", [([40], 0), ([40], 111), ([2], 111), ([40], 250), ([1], 0)])
def test_one_page_of_a_short_cache(page, new, window):
    """300 tokens; with the window of 111 the first row of 40 sees from place 150 on."""
    pages = -(-300 // page)
    for gone in range(0, pages, max(1, pages // 8)):
        check(new, [300], 4, 2, 128, page, "bf16", window=window, change=without(gone))


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("D,n", [(128, 4950), (64, 3200)])
def test_one_page_of_a_cache_that_several_ctas_walk(page, D, n):
    """70 tokens behind a long context: too few rows to fill the device."""
    pages = -(-n // page)
    for gone in range(0, pages, max(1, pages // 20)):
        check([70], [n], 4, 2, D, page, "fp16", change=without(gone))


@pytest.mark.parametrize("page", [128, 256])
def test_several_pages_of_prompts(page):
    def change(q, cache, table, kv):
        table[0, 0] = table[0, 3] = table[1, 1] = -5
        table[2] = -1
    check([300, 129, 40, 5], [1300, 600, 400, 300], 6, 2, 128, page, "bf16", window=333, scales=True, pad=3, change=change)
