"""B200-native (sm_100a) chunkwise Gated DeltaNet layer, forward and backward, and two
operators around it: the gated linear recurrence and the q/k normalisation with rotation.

The compute lives in libgdn.so (CUDA kernels behind the C ABI in
include/gdn.h); this package is its thin Python binding plus the seeded
synthetic-input generator.  Importing it does not load the library; the first
call does, and raises if the library was not built.
"""
from ._binding import (EXPORTS, GDN_BF16, GDN_FLAG_PIECE_SCAN, GDN_FLAG_QK_L2NORM,  # noqa
                       GDN_FLAG_VALUE_SLICES, GDN_FP32, GDN_LINREC_COMPLEMENT, GDN_NORM_L2,
                       GDN_NORM_NONE, GDN_NORM_RMS, GDN_QK_INTERLEAVED,
                       GDN_TEST_FAIL_LAUNCH, GDN_TEST_STALL_COPY, GdnDesc, GdnError, GdnLinrecDesc, GdnQkDesc, LaunchTrace,
                       alloc_workspace, bwd_workspace_size, device_status, fwd_workspace_size,
                       gdn_bwd, gdn_decode, gdn_fwd, gdn_linrec_bwd, gdn_linrec_decode,
                       gdn_linrec_fwd, gdn_qk_norm_rope_bwd, gdn_qk_norm_rope_fwd, lib,
                       linrec_status, make_desc, set_test_hook,
                       set_wait_limit)

__all__ = ["gdn_fwd", "gdn_bwd", "gdn_decode", "gdn_linrec_fwd", "gdn_linrec_bwd",
           "gdn_linrec_decode", "linrec_status", "gdn_qk_norm_rope_fwd", "gdn_qk_norm_rope_bwd", "device_status", "fwd_workspace_size",
           "bwd_workspace_size", "alloc_workspace", "LaunchTrace", "make_desc", "GdnDesc",
           "GdnError", "lib", "GDN_BF16", "GDN_FP32", "GDN_FLAG_PIECE_SCAN", "GDN_FLAG_QK_L2NORM",
           "GDN_FLAG_VALUE_SLICES", "GDN_LINREC_COMPLEMENT", "GdnLinrecDesc", "GDN_NORM_NONE",
           "GDN_NORM_L2", "GDN_NORM_RMS", "GDN_QK_INTERLEAVED", "GdnQkDesc",
           "GDN_TEST_STALL_COPY", "GDN_TEST_FAIL_LAUNCH", "set_wait_limit", "set_test_hook",
           "EXPORTS"]
