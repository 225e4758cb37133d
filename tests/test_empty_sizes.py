"""CPU check of the workspace sizes of weights with no rows or no columns, at row counts on
both sides of every path's limit: a size that serves the call (which then does nothing), and
no division by a number of tiles that is zero.  In a process of its own, since such a
division ends the process."""
import subprocess
import sys

QUERIES = """
import ctypes
import itertools
import int4_w4a16_group_g32_amd as L

lib, r = L.load_library(), ctypes.byref


def desc(K, N, E=1):
    return L.WeightDesc(0x100000, 0x200000, K, N, 32, E, L.LAYOUT_GROUPED)


lo = [L.LoraDesc(0x300000, 0x400000, 0x500000, None, rank, 4) for rank in (16, 256)]
n = 0
for M, xt, (K, N), lora in itertools.product((1, 8, 9, 16, 17, 20, 64, 65, 100, 256, 512, 513, 600, 2 ** 31 - 1),
                                             (L.F32, L.BF16), ((0, 128), (64, 0), (0, 0), (0, 64), (128, 0)), lo):
    w, d, e, f = desc(K, N), desc(N, K), desc(K, N, 6), desc(N, K, 6)
    got = [lib.w4a16_gemm_workspace_bytes(M, r(w), xt), lib.w4a16_swiglu_mlp_workspace_bytes(M, xt, r(w), r(w), r(d)),
           lib.w4a16_gemm_lora_workspace_bytes(M, r(w), xt, r(lora)),
           lib.w4a16_swiglu_mlp_lora_workspace_bytes(M, xt, r(w), r(w), r(d), r(lora), None, r(lora))]
    if M < 1 << 20:
        got.append(lib.w4a16_moe_workspace_bytes(M, 2, xt, r(e), r(e), r(f)))
        got.append(lib.w4a16_moe_shared_workspace_bytes(M, 2, xt, r(e), r(e), r(f), r(w), r(w), r(d)))
    if M <= (8 if xt == L.F32 else 16):
        got.append(lib.w4a16_moe_decode_workspace_bytes(M, 2, xt, r(e), r(e), r(f), None, None, None))
        got.append(lib.w4a16_moe_decode_workspace_bytes(M, 2, xt, r(e), r(e), r(f), r(w), r(w), r(d)))
    assert all(v > 0 for v in got), (M, xt, K, N, got)
    n += len(got)
print("sizes", n)
"""


def test_sizes_of_empty_weights():
    p = subprocess.run([sys.executable, "-c", QUERIES], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, f"exit {p.returncode}: {p.stderr[-500:]}"
    assert p.stdout.startswith("sizes ")
