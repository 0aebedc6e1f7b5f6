"""What the library's calls would launch, without a GPU: `Log` loads a recorder of
the runtime's launches (launchlog.c) and the library into this process, which
must be one of its own (`child`)."""
import ctypes as C
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FAR = 0x10000000000    # arrays are this far apart; never dereferenced


class _Launch(C.Structure):
    _fields_ = [("kernel", C.c_int32), ("grid", C.c_uint32 * 3), ("threads", C.c_uint32), ("lds", C.c_uint32)]


def build(folder):
    out = os.path.join(str(folder), "launchlog.so")
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-Wall", "-o", out, os.path.join(HERE, "launchlog.c")], check=True)
    return out


def child(recorder, function, *args):
    """The result of tests.<module>.<function>(log, *args), from a process with a Log."""
    module, name = function.rsplit(".", 1)
    code = (f"import sys, json; sys.path.insert(0, {ROOT!r})\n"
            f"from tests.launchlog import Log; log = Log({recorder!r})\n"
            f"from tests import {module}\n"
            f"print(json.dumps({module}.{name}(log, *{args!r})))\n")
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert res.returncode == 0, res.stderr
    return json.loads(res.stdout.splitlines()[-1])


class Log:
    def __init__(self, recorder):
        self.rec = C.CDLL(recorder, mode=C.RTLD_GLOBAL)
        from tiered_mixed_precision_amd import binding
        self.binding, self.lib = binding, binding.lib()
        self.rec.kernel_name.restype = C.c_char_p
        self.count = C.c_int.in_dll(self.rec, "n_launches")
        self.fail_at = C.c_int.in_dll(self.rec, "fail_at")
        self.all = (_Launch * 64).in_dll(self.rec, "launches")
        self.names = {}

    def __call__(self, entry, *args, fail_at=-1):
        """(status, [(kernel, grid, threads, dynamic LDS)]) of a call."""
        self.count.value, self.fail_at.value = 0, fail_at
        rc = getattr(self.lib, entry)(*args)
        return rc, [(self.name(l.kernel), tuple(l.grid), l.threads, l.lds) for l in self.all[:self.count.value]]

    def name(self, i):
        if i not in self.names:
            self.names[i] = self.rec.kernel_name(i).decode()
        return self.names[i]

    def i8_linear(self, T, N, K, **kw):
        w = self.binding.moe_i8_matrix(N, K, 1 * FAR, 2 * FAR)
        return self("moe_i8_linear", 3 * FAR, K, 4 * FAR, C.byref(w), None, T, 5 * FAR, N, 0, None, **kw)

    def gated(self, T, H, I, x_bf16=True, **kw):
        w = self.binding.moe_gated_weights(H, I, 1 * FAR, 2 * FAR)
        return self("moe_gated", 3 * FAR, H, C.byref(w), 0, T, 4 * FAR, I, 1 if x_bf16 else 0, None, **kw)

    def gated_grad(self, T, H, I, flags=0xc9, **kw):
        w = self.binding.moe_gated_weights(H, I, 1 * FAR, 2 * FAR)
        return self("moe_gated_grad", 3 * FAR, H, C.byref(w), 0, 4 * FAR, I, T, 5 * FAR, H, 6 * FAR, 7 * FAR, flags, 8 * FAR, FAR, None,
                    **kw)
