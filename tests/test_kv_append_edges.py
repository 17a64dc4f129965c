"""pa_kv_append and pa_kv_append_q8: what a promise of the language, a tie or an empty argument decides."""
import os
import re


def test_what_the_append_writes_is_not_loaded_as_constant(cuda_lib):
    """__ldg promises that its array stays as it is during the launch: none that the appends write is loaded so."""
    csrc = os.path.join(os.path.dirname(cuda_lib.LIB_PATH), "csrc")
    with open(os.path.join(csrc, "pa_append.cu")) as f:
        text = f.read()
    for name in ("k_scales", "v_scales", "key_cache", "value_cache", "query_out"):
        assert not re.search(r"__ldg\([^;]*\b%s\b" % name, text), name
