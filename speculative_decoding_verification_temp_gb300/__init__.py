"""GB300-native speculative-sampling verification.

The computation lives in libspecverify.so (CUDA for sm_103a, C ABI declared
in include/specverify.h); ``api`` is a thin torch binding over it.

  verify_chain   accept drafts with probability min(1, p/q), stop at the first
                 rejection, draw the correction from norm([p - q]+) or a bonus
                 token from p
  verify_tree    recursive rejection over sibling candidates of token trees
  tree_mask      ancestor-or-self attention masks and depth position ids
  overlap        per-position acceptance rate beta_i = sum_v min(p_i, q_i)
  typical_accept typical acceptance (entropy threshold; approximate, not
                 distribution-exact)
  tree_rerank    EAGLE-2 rerank: the top-m nodes of a draft tree by path value

and the paged key-value cache around it (``cache``):

  paged_attention  attention of new tokens (one, a chain, a tree) over a cache's
                   pages, with a sliding window and sinks
  cache_append     new tokens' keys and values into the pages
  cache_compact    a tree's accepted path moved together
  cache_resize     pages taken for, or given back behind, a length
  cache_fork       sequences that go on from another one's tokens
  cache_read       tokens of the pages back as rows
  cache_4bit       a cache of 4-bit rows, which all of these take
  rotary           queries and keys rotated by their positions (rotary_frequency:
                   plain or scaled frequencies)
  cache_append_rotary  new queries and keys rotated, keys and values into the pages
"""

from ._abi import (FLAG_BAD_LENGTH, FLAG_BAD_PAGE, FLAG_BAD_SEQUENCE, FLAG_BAD_TOKEN,  # noqa: F401
                   FLAG_BAD_TREE, FLAG_DEGENERATE_RESIDUAL, FLAG_DEPTH, FLAG_NO_PAGES,
                   FLAG_NONFINITE, FLAG_TIMEOUT, FLAG_ZERO_Q)


def __getattr__(name):
    # the torch binding is imported on first use, so the workload generator
    # and the build step do not need torch
    if name in ("verify_chain", "verify_chain_static", "verify_tree", "tree_mask", "overlap",
                "typical_accept", "tree_rerank", "SpecVerifyError", "workspace",
                "ChainResult", "TreeResult", "MaskResult", "OverlapResult", "TypicalResult",
                "RerankResult", "set_wait_limit", "api"):
        import importlib
        api = importlib.import_module(__name__ + ".api")
        return api if name == "api" else getattr(api, name)
    if name in ("paged_attention", "cache_append", "cache_compact", "cache_resize", "cache_fork",
                "cache_read", "cache_4bit", "cache_append_rotary", "rotary", "rotary_frequency",
                "RotaryAppendResult", "ReadResult", "RotaryFrequency", "page_pool", "PagePool", "AttentionResult", "CompactResult", "cache"):
        import importlib
        cache = importlib.import_module(__name__ + ".cache")
        # importlib binds the module to the name `cache`; the functions are bound
        # here, so that later uses do not come through this function
        globals()[name] = found = cache if name == "cache" else getattr(cache, name)
        return found
    raise AttributeError(name)
