"""The training entry points replaced by functions that wait for another thread of Python,
so that a call through the native binding ends well only if it lets that thread run.
They launch nothing and give up after some seconds."""
import os
import subprocess
import sys

ENTRIES = ["moe_balance_loss", "moe_route_backward", "moe_gemm_fp8", "moe_gemm_fp8_dgrad", "moe_quantize_act_fp8",
           "moe_quantize_fp8_tokens", "moe_gemm_fp8_wgrad"]

_C = """
#include <unistd.h>
static volatile int inside, released;
int stub_inside(void) { return inside; }
void stub_release(void) { released = 1; }
static int hold(void) {
    inside = 1;
    int i;
    for (i = 0; i < 4000 && !released; ++i) usleep(1000);
    inside = 0;
    const int code = released ? 0 : 5;
    released = 0;
    return code;
}
"""

_DRIVER = """
import ctypes, os, sys, threading, time
import torch
import expert_layer_dual_b200.moe as M
stub = ctypes.CDLL(os.environ["LD_PRELOAD"])

def call(name, *args):
    def release():
        for _ in range(20000):
            if stub.stub_inside():
                return stub.stub_release()
            time.sleep(0.001)
    t = threading.Thread(target=release)
    t.start()
    status = getattr(M._native, name)(*args)
    t.join()
    print(name, status)
"""


def run(tmp_path, calls):
    """{entry: status} of the lines of `calls`, `call(name, arguments of the native entry)`."""
    src, lib = os.path.join(tmp_path, "stub.c"), os.path.join(tmp_path, "libstub.so")
    with open(src, "w") as f:
        f.write(_C + "".join(f"int {e}() {{ return hold(); }}\n" for e in ENTRIES))
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", src, "-o", lib], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _DRIVER + calls], cwd=root, capture_output=True, text=True, timeout=240,
                       env={**os.environ, "LD_PRELOAD": lib})
    assert r.returncode == 0, r.stderr[-2000:]
    return {line.split()[0]: int(line.split()[1]) for line in r.stdout.splitlines()}
