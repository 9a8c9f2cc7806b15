"""Host side of the convolution, the scan and the norms at the limits of their sizes: nothing is launched."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

from chunked_gated_delta_06_gb300 import binding, build

MOST = (1 << 31) - 65536   # tokens of a pack


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.lib()


def _pack(*lens):
    host = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    p = binding.GdnPack(len(host) - 1, int(host[-1]), host.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), 0x10000, None)
    p.keep = host
    return p


def _scan_bytes(lens, channels=1, state_dim=8, segment=0, backward=0):
    s = binding.GdnScanShape(channels, 1, state_dim, binding.GDN_DTYPE_BF16, 0, 0, 0, 0, 0, segment)
    return binding.lib().gdn_selective_scan_workspace_bytes(ctypes.byref(_pack(*lens)), ctypes.byref(s), backward)


# (the library's plan tries longer and longer segments; in a process of its own, as one that does not end, or a
# division by zero, ends the process)
@pytest.mark.parametrize("lens", [(1 << 30,), ((1 << 30) + 1,), (MOST,), (100, (1 << 30) + 100, 0, 7)])
def test_sequences_up_to_the_longest_have_a_plan(lens):
    call = "import test_mixer_limits as t; print(*[t._scan_bytes(%r, backward=b) for b in (0, 1)])" % (lens,)
    out = subprocess.run([sys.executable, "-c", call], cwd=os.path.dirname(os.path.abspath(__file__)), capture_output=True,
                         text=True, timeout=60, env={**os.environ, "PYTHONPATH": os.path.dirname(build.PKG)})
    assert out.returncode == 0, (out.returncode, out.stderr)
    fwd, bwd = map(int, out.stdout.split())
    # one channel of 8 states: one record of a segment is 36 bytes at least, marks of 32 bytes for each 8 tokens
    assert fwd >= 36 and bwd >= sum(lens) // 8 * 32


def test_rows_of_a_step_that_indices_do_not_hold_are_refused(lib):
    # (what fits the check goes on to the launch, which this machine may have no device for: not made here)
    bf, bad, fake = binding.GDN_DTYPE_BF16, binding.GDN_ERR_INVALID_ARG, [(i + 1) << 40 for i in range(12)]
    s = binding.GdnScanShape(1, 1, 8, bf, 0, 0, 0, 0, 0, 0)
    for batch in (MOST + 1, (1 << 31) - 32, (1 << 31) - 1):
        assert lib.gdn_short_conv_step(batch, 1, 4, 1, bf, fake[0], 1, fake[1], None, fake[2], 4, fake[3], fake[4], None, None) == bad
        assert lib.gdn_selective_scan_step(batch, ctypes.byref(s), *fake[:5], None, None, None, fake[5], 4, fake[6], fake[7], None,
                                           None) == bad


def test_parameters_start_where_the_header_says(lib):
    # the convolution's and the scan's on their element's size, the norms' on 16 bytes (each call with a workspace
    # too small or an output over an input, so that none gets as far as a launch)
    bf, bad, small = binding.GDN_DTYPE_BF16, binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_WORKSPACE_TOO_SMALL
    at = [(i + 1) << 30 for i in range(24)]
    p, s = ctypes.byref(_pack(9)), ctypes.byref(binding.GdnScanShape(8, 1, 8, bf, 0, 0, 0, 0, 0, 0))
    for off in (0, 4):
        q = [a + off for a in at]   # parameters and their gradients
        assert lib.gdn_short_conv_bwd(p, 8, 4, 1, bf, at[0], 8, q[1], q[2], None, at[3], None, at[4], q[5], q[6], None, at[7], 0,
                                      None) == small
        assert lib.gdn_selective_scan_bwd(p, s, at[0], at[1], q[2], at[3], at[4], q[5], None, q[6], None, at[7], None, at[8], at[9],
                                          q[10], at[11], at[12], q[13], None, q[14], None, at[15], 0, None) == small
    norm = lambda weight, scale, dw, ds: lib.gdn_rms_norm_bwd(  # noqa: E731
        4, 128, bf, bf, 0, 1e-6, 0.0, at[0], at[1], scale, weight, None, at[2], None, at[3], at[4], None, dw, ds, at[5], 0, None)
    assert norm(at[6], at[7], at[8] + 4, at[9] + 4) == small
    assert norm(at[6] + 4, at[7], at[8], at[9]) == norm(at[6], at[7] + 4, at[8], at[9]) == bad


@pytest.mark.parametrize("lens, channels, state_dim", [((300, 0, 150), 96, 16), ((500, 260), 160, 8), ((700, 33), 96, 32),
                                                       ((5000,), 32, 16), ((65536,), 2048, 16)])
def test_long_sequences_of_few_channels_are_split(lens, channels, state_dim):
    for back in (0, 1):
        plan, whole = (_scan_bytes(lens, channels, state_dim, s, back) for s in (0, -1))
        assert plan > whole, back


def test_calls_of_few_tokens_are_not_split():
    # (the Python calls of up to 64 tokens ask for no workspace first)
    for lens in ((1,), (32,), (33,), (64,), (0, 63, 1), (33, 31), (1,) * 64):
        for channels in (1, 17, 2048, 1 << 16, 1 << 20):
            for state_dim in (8, 16, 32):
                assert _scan_bytes(lens, channels, state_dim) == 256
