"""Test builds of the library that differ in a few translation units: those
are compiled with other constants and linked with the regular build's
objects."""
import os
import subprocess

from paged_quantized_kv_gb300 import build as kbuild


def build_variant(folder, units):
    """units: {source: {constant: value}}; returns the library's path."""
    objects = {s: os.path.join(kbuild.BUILD, s.replace(".cu", ".o"))
               for s in kbuild.SOURCES}
    kbuild.build(force=not all(map(os.path.exists, objects.values())))
    nvcc, jobs = kbuild._nvcc(), []
    for source, constants in units.items():
        objects[source] = os.path.join(str(folder),
                                       source.replace(".cu", ".o"))
        jobs.append(subprocess.Popen(
            [nvcc, *kbuild.ARCH, *kbuild.NVCC_FLAGS,
             *[f"-D{k}={v}" for k, v in constants.items()], "-c",
             os.path.join(kbuild.CSRC, source), "-o", objects[source]]))
    assert all(j.wait() == 0 for j in jobs)
    out = os.path.join(str(folder), "libkvq_variant.so")
    subprocess.run([nvcc, *kbuild.ARCH, "-shared", "-cudart", "static",
                    *objects.values(), "-o", out], check=True)
    return out
