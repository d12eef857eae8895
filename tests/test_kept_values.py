"""Source check: what the host code keeps from one call for the next (occupancies, functions
already set up, per device) is atomic, since calls from several threads may fill it at once."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_mixed_precision_gb300", "csrc")


def test_kept_values_are_atomic():
    found = []
    for name in sorted(os.listdir(CSRC)):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        # tables per device, and function-local statics that are not constants
        found += [(name, m[0]) for m in re.finditer(r"^[^\n;(]*\w+\[64\](?:\s*=[^;]*)?;", src, re.M)
                  if "std::atomic" not in m[0] and re.match(r"\s*(static\s+)?(int|bool)\b", m[0])]
        found += [(name, m[0]) for m in re.finditer(r"^\s+static (?!const|std::atomic|thread_local|inline|__device__)[^;()]*(?:=[^;]*)?;", src, re.M)
                  if "constexpr" not in m[0]]
    assert not found, found
