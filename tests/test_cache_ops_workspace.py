"""Sizes of the page operators' workspace (no GPU is needed)."""
import moe_token_dispatch_persistent_gb300 as mk
from moe_token_dispatch_persistent_gb300 import build as mkbuild


def test_pages_workspace_does_not_grow_with_the_rows_of_a_table():
    mkbuild.build()
    for pages, n in ((20, 4096), (1 << 20, 7), (0, 0)):
        assert mk.mk_pages_workspace_size(2 ** 31 - 1, pages, n) == mk.mk_pages_workspace_size(1, pages, n)
        assert mk.mk_pages_workspace_size(1, pages, n) <= 12 * pages + 8 * n + 8192
