// csrc/per_device.h with devices and outcomes of the test's choice (tests/test_per_device.py).
#include "per_device.h"

static coli::PerDevice state;

// the status of a call on `device` whose set would return `outcome`; *ran: was it called?
extern "C" int once_on(int device, int outcome, int *ran) {
  *ran = 0;
  return state.once(device, [&]() {
    *ran = 1;
    return outcome;
  });
}
